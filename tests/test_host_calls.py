"""What a call does on the host around its launches, without a GPU: the
library and its binding run against a stand-in for HIP's launch and device
calls (tests/native/hip_stub.cpp), in a process of their own."""
import os
import subprocess
import sys
import textwrap

import pytest

from bit_weight_quantized_awq_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    """The stand-in, built."""
    path = str(tmp_path_factory.mktemp("stub") / "hip_stub.so")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.hipcc()))), "include")
    cmd = ["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-isystem",
           include, os.path.join(ROOT, "tests", "native", "hip_stub.cpp"), "-o", path]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return path


PRELUDE = """
import ctypes, sys, threading
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
stub.stub_thread.restype = ctypes.c_uint64
"""


def run(stub, program):
    """Runs `program` after the stand-in has been loaded; it prints "ok"."""
    res = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(program), stub], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.endswith("ok\n"), res.stdout + res.stderr


def test_calls_that_share_a_workspace_are_not_interleaved(stub):
    """Kernels of a call that hand each other data through the workspace are
    launched one after the other, whatever other host threads launch."""
    run(stub, """
        import bit_weight_quantized_awq_amd as awq
        from bit_weight_quantized_awq_amd import binding as b
        A, WS = 0x10000, 0x100000
        c = b.KvCacheStruct(k=A, v=A, num_blocks=1000, block_size=16, heads=8, head_dim=128,
                            k_block_stride=16384, k_slot_stride=1024, k_head_stride=128,
                            v_block_stride=16384, v_slot_stride=1024, v_head_stride=128)
        lib = awq.lib()

        def attention():     # the kernel and the join
            return lib.awq_tree_attention(A, ctypes.byref(c), A, A, A, None, A, 2, 4, 32, 100, 100,
                                          0, 4096, 128, 0.1, b.AWQ_F16, WS, 1 << 40, None)

        def product():       # split along K, and the sum
            return lib.awq_gemm(A, A, A, A, None, A, 16, 14336, 4096, 128, WS, 1 << 40, None)

        def gathered():      # the reordered x, the product and its sum
            return lib.awq_gemm_sorted(A, A, A, A, A, None, A, 128, 4096, 4096, 4096, 128, WS,
                                       1 << 40, None)

        for f, n in ((attention, 2), (product, 2), (gathered, 3)):
            stub.stub_clear()
            assert f() == 0 and stub.stub_launches() == n, (f.__name__, stub.stub_launches())

        stub.stub_clear()
        calls = {attention: 2, product: 2, gathered: 3}
        names, failed = {}, []

        def work(f):
            names[threading.get_ident()] = calls[f]
            for _ in range(40):
                if f() != 0:
                    failed.append(f)

        threads = [threading.Thread(target=work, args=(f,)) for f in calls for _ in range(2)]
        for t in threads: t.start()
        for t in threads: t.join()
        assert not failed
        order = [stub.stub_thread(i) for i in range(stub.stub_launches())]
        assert len(order) == 2 * 40 * 7
        i = 0
        while i < len(order):
            n = names[order[i]]
            assert order[i:i + n] == [order[i]] * n, (i, order[i:i + n])
            i += n
        print("ok")
        """)


DEVICES = """
import torch
# Tensors of two devices that are not there, in host memory.
torch.cuda._initialized = True
torch.cuda.memory.change_current_allocator(
    torch.cuda.memory.CUDAPluggableAllocator(sys.argv[1], "stub_alloc", "stub_free"))
import bit_weight_quantized_awq_amd as awq
F16, I32, I64 = torch.float16, torch.int32, torch.int64

def new(*shape, dtype=I32, device="cuda:1"):
    return torch.empty(shape, dtype=dtype, device=device)

def on_one(call, launches=1):
    # A call on tensors of device 1, with device 0 current.
    assert torch.cuda.current_device() == 0
    stub.stub_clear()
    call()
    seen = [stub.stub_device(i) for i in range(stub.stub_launches())]
    assert seen == [1] * launches, seen
    assert torch.cuda.current_device() == 0
"""


def test_serving_calls_launch_on_their_tensors_device(stub):
    run(stub, DEVICES + textwrap.dedent("""
        k, q, cache = new(4, 2, 64, dtype=F16), new(4, 8, 64, dtype=F16), new(10, 16, 2, 64, dtype=F16)
        two, three = new(2), new(3)
        on_one(lambda: awq.batch_layout(two, two, two, new(5), new(2, 4), 16, 10, 4))
        on_one(lambda: awq.kv_write(k, k, new(4), cache, cache))
        ws = new(1 << 24, dtype=torch.uint8)
        on_one(lambda: awq.tree_attention(q, cache, cache, new(2, 400), two, three, workspace=ws), 2)
        on_one(lambda: awq.process_logits(new(4, 500, dtype=F16)))
        print("ok")
        """))


def test_linear_calls_launch_on_their_tensors_device(stub):
    run(stub, DEVICES + textwrap.dedent("""
        K, N, g = 256, 128, 64
        x, w = new(2, K, dtype=F16), new(K, N // 8)
        z, s, y = new(K // g, N // 8), new(K // g, N, dtype=F16), new(2, N, dtype=F16)
        ws, gidx = new(1 << 24, dtype=torch.uint8), new(K)
        on_one(lambda: awq.gemm(x, w, z, s, None, g, workspace=ws))
        # The first one clears the scratch of its device.
        on_one(lambda: awq.gemm_noalloc(x, w, z, s, None, g), 2)
        on_one(lambda: awq.gemm_noalloc(x, w, z, s, None, g))
        on_one(lambda: awq.dequant(w, z, s, g))
        on_one(lambda: awq.dequant_gidx(w, z, s, gidx))
        on_one(lambda: awq.gemm_gidx(x, w, z, s, gidx))
        on_one(lambda: awq.gather_rows(w, new(5)))
        on_one(lambda: awq.dense_gemv(x, new(N, K, dtype=F16)))
        # The x that a batch of 64 rows reorders, and the product.
        sorted_w = awq.SortedWeight(w, z, s, gidx, g, K)
        on_one(lambda: awq.gemm_sorted(new(64, K, dtype=F16), sorted_w, workspace=ws), 2)
        print("ok")
        """))


def test_tensors_without_memory_raise(stub):
    """Operands that hold no memory (fake ones, as tracers make them) end in
    an exception, not in a process without the interpreter's lock."""
    run(stub, DEVICES + textwrap.dedent("""
        def none(*shape, dtype=I32):
            t = new(*shape, dtype=dtype)
            torch._C._set_throw_on_mutable_data_ptr(t)
            return t

        k, q, cache = new(4, 2, 64, dtype=F16), new(4, 8, 64, dtype=F16), new(10, 16, 2, 64, dtype=F16)
        two, three, table = new(2), new(3), new(2, 4)
        ws = new(1 << 24, dtype=torch.uint8)
        for call in [
                lambda: awq.batch_layout(none(2), two, two, new(5), table, 16, 10, 4),
                lambda: awq.batch_layout(two, two, two, new(5), none(2, 4), 16, 10, 4),
                lambda: awq.kv_write(none(4, 2, 64, dtype=F16), k, new(4), cache, cache),
                lambda: awq.kv_write(k, k, none(4), cache, cache),
                lambda: awq.kv_write(k, k, new(4), none(10, 16, 2, 64, dtype=F16), cache),
                lambda: awq.tree_attention(none(4, 8, 64, dtype=F16), cache, cache, table, two, three,
                                           workspace=ws),
                lambda: awq.tree_attention(q, cache, cache, none(2, 4), two, three, workspace=ws),
                lambda: awq.tree_attention(q, cache, cache, table, two, none(3), workspace=ws),
                lambda: awq.tree_attention(q, cache, cache, table, two, three,
                                           workspace=none(1 << 24, dtype=torch.uint8)),
                lambda: awq.process_logits(none(4, 500, dtype=F16)),
                lambda: awq.process_logits(new(4, 500, dtype=F16), requests=none(4))]:
            stub.stub_clear()
            try:
                call()
            except RuntimeError as e:
                pass
            else:
                raise AssertionError("no exception")
            assert stub.stub_launches() == 0
            assert torch.cuda.current_device() == 0
        on_one(lambda: awq.kv_write(k, k, new(4), cache, cache))
        print("ok")
        """))


def test_masks_of_no_words_are_refused(stub):
    """A mask that has no bits is no causal chain."""
    run(stub, DEVICES + textwrap.dedent("""
        q, cache = new(4, 8, 64, dtype=F16), new(10, 16, 2, 64, dtype=F16)
        ws = new(1 << 24, dtype=torch.uint8)
        stub.stub_clear()
        try:
            awq.tree_attention(q, cache, cache, new(2, 4), new(2), new(3), tree_mask=new(4, 0, dtype=I64),
                               workspace=ws)
        except ValueError as e:
            assert "tree_mask" in str(e)
        else:
            raise AssertionError("no exception")
        try:
            awq.process_logits(new(4, 50, dtype=F16), requests=new(4), draft_tokens=new(4),
                               tree_mask=new(4, 0, dtype=I64), q_start=new(3))
        except ValueError as e:
            assert "tree_mask" in str(e)
        else:
            raise AssertionError("no exception")
        assert stub.stub_launches() == 0
        print("ok")
        """))


def test_refusals_say_what_serving_calls_refuse(stub):
    """The texts of the statuses name the limits of these calls, too."""
    run(stub, DEVICES + textwrap.dedent("""
        import re
        q, cache = new(4, 8, 96, dtype=F16), new(10, 16, 2, 96, dtype=F16)
        small = new(16, dtype=torch.uint8)
        good, fine = new(4, 8, 64, dtype=F16), new(10, 16, 2, 64, dtype=F16)
        shifted = torch.empty(4 * 8 * 64 + 1, dtype=F16, device="cuda:1")[1:].view(4, 8, 64)
        for call, words in [
                (lambda: awq.tree_attention(q, cache, cache, new(2, 4), new(2), new(3), workspace=small),
                 "head_dim"),
                (lambda: awq.tree_attention(good, fine, fine, new(2, 4), new(2), new(3), workspace=small),
                 "awq_tree_attention_workspace_size"),
                (lambda: awq.tree_attention(shifted, fine, fine, new(2, 4), new(2), new(3),
                                            workspace=small), "16 bytes"),
                (lambda: awq.tree_attention(good, fine, fine, new(2, 4), new(2), new(3), scale=1e39,
                                            workspace=small), "finite")]:
            try:
                call()
            except awq.AwqError as e:
                assert words in str(e), (words, str(e))
            else:
                raise AssertionError("no exception")
        print("ok")
        """))
