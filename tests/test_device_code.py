"""The assembly of the kernels whose memory instructions are written inline:
the compiler adds the wait states that the hardware asks for between its own
instructions only."""
import os
import re
import subprocess

import pytest

from bit_weight_quantized_awq_amd import build


def instructions(source, tmp_path):
    """The device code of a source under csrc/, one instruction or label each."""
    out = str(tmp_path / "device.s")
    cmd = ([build.hipcc(), "-x", "hip", "-S", "--cuda-device-only",
            os.path.join(build.CSRC, source), "-o", out] + build.COMMON_FLAGS +
           build.FILE_FLAGS.get(source, []))
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    with open(out) as f:
        lines = [line.split(";")[0].strip() for line in f]
    return [x for x in lines if x and (x.endswith(":") or not x.startswith("."))]


def scalar_registers(operands):
    found = set()
    for first, last, single in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", operands):
        found |= {int(single)} if single else set(range(int(first), int(last) + 1))
    return found


@pytest.mark.parametrize("source", ["awq_prefill.hip", "awq_attention.hip"])
def test_wait_states_before_memory_instructions(source, tmp_path):
    """One wait state from a scalar write of m0 to a copy to LDS, whose
    address it is; five from a vector instruction that writes a scalar
    register (a lane read) to a memory instruction that reads it."""
    code = instructions(source, tmp_path)
    copies, early = 0, []
    for i, x in enumerate(code):
        op, _, operands = x.partition(" ")
        if not op.startswith(("buffer_", "global_", "flat_", "scratch_")):
            continue
        copy = op.startswith("global_load_lds") or operands.endswith(" lds")
        copies += copy
        used, waited = scalar_registers(operands), 0
        for before in reversed(code[max(0, i - 8):i]):
            name, _, rest = before.partition(" ")
            if name.endswith(":"):
                continue
            if name == "s_nop":
                waited += int(rest, 0) + 1
            else:
                written = rest.split(",")[0]
                if copy and waited < 1 and name.startswith("s_") and written.strip() == "m0":
                    early.append((before, x))
                if name.startswith("v_") and scalar_registers(written) & used:
                    early.append((before, x))
                waited += 1
            if waited >= 5:
                break
    assert copies > 100
    assert not early, (len(early), early[:5])
