"""The serving pass's host code, and the one kernel whose lengths decide its
addresses, built for the CPU and run under AddressSanitizer and UBSan."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_weight_quantized_awq_amd", "csrc")
NATIVE = os.path.join(ROOT, "tests", "native")
CXX = shutil.which("g++")


def run_checked(tmp_path, name, sources, includes):
    """Builds `sources` with the sanitizers and returns the program's output."""
    if CXX is None:
        pytest.skip("g++ is needed")
    exe = str(tmp_path / name)
    cmd = [CXX, "-std=c++17", "-O1", "-g", "-pthread", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Wno-unknown-pragmas", "-Wno-unused-function",
           *(f"-I{d}" for d in includes), *sources, "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    return res.stdout


def test_layout_kernel_where_sums_pass_32_bits(tmp_path):
    """awq_batch_layout's kernel on the CPU: no access leaves the operands
    whatever the lengths hold, and sums past 2^31 - 1 are held there."""
    with open(os.path.join(CSRC, "awq_layout.hip")) as f:
        text = f.read()
    # The operators' launch entry, and dynamic shared memory, as the CPU has them.
    for old, new in (('#include "awq_device.h"', '#include "gpu_on_cpu.h"'),
                     ("extern __shared__ int32_t smem[];",
                      "int32_t* smem = gpu_on_cpu::lds.data();")):
        assert text.count(old) == 1, old
        text = text.replace(old, new)
    (tmp_path / "layout_kernel_source.h").write_text(text)
    out = run_checked(tmp_path, "layout_check", [os.path.join(NATIVE, "layout_check.cpp")],
                      [str(tmp_path), NATIVE, CSRC, os.path.join(ROOT, "include")])
    assert "layout_check ok" in out


def test_validation_and_planning(tmp_path):
    """The checks of arguments, and what a plan writes against the workspace
    it asks for, over extreme sizes."""
    out = run_checked(tmp_path, "verify_check",
                      [os.path.join(NATIVE, "verify_check.cpp"), os.path.join(CSRC, "awq_verify.cpp"),
                       os.path.join(CSRC, "awq_plan.cpp")], [CSRC, os.path.join(ROOT, "include")])
    assert "verify_check ok" in out
