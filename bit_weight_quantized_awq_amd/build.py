"""Build the C-ABI shared library libawq_mi355x.so for gfx950 with hipcc.

Every source of the library under csrc/ is compiled as HIP for gfx950 into
_build/, then linked into the package directory, where the Python binding
loads it from.  Packed fp32 VALU instructions are disabled in device code.
A second, separate library, libawq_bench.so (csrc/bench_read.hip: a plain
read stream that the benchmark uses as a same-box reference), is built the
same way; the W4A16 path never loads it.  _serving.so (csrc/serving_bind.cpp,
host code against torch's headers, left out where torch is missing) is the
Python module behind serving.py; it links the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libawq_mi355x.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BENCH_LIB_PATH = os.path.join(PKG_DIR, "libawq_bench.so")
BENCH_SOURCES = ["bench_read.hip"]
BIND_PATH = os.path.join(PKG_DIR, "_serving.so")
BIND_SOURCE = "serving_bind.cpp"
ARCH = "gfx950"

SOURCES = [
    "awq_plan.cpp",
    "awq_api.cpp",
    "awq_dequant.hip",
    "awq_generic.hip",
    "awq_decode.hip",
    "awq_prefill.hip",
    "awq_dense.hip",
    "awq_gidx.hip",
    "awq_verify.cpp",
    "awq_verify_api.cpp",
    "awq_layout.hip",
    "awq_cache.hip",
    "awq_attention.hip",
    "awq_logits.hip",
]

COMMON_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}",
    f"-I{CSRC}",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain (ROCm) is required to build")


# Per-file flags.  The decode kernels are short (about 9 us), so the start
# of every wave counts: their first kernel arguments are preloaded into
# SGPRs at wave launch instead of being fetched from the argument segment by
# the first instructions (a code-object feature of gfx950; the kernel keeps
# a fallback prologue that fetches them itself when the launcher does not
# preload).  Same box, K=8192 N=7168: M=1 9.375 -> 9.316 us, M=16 13.47 ->
# 13.34 us; K=14336 N=4096 M=1 9.566 -> 9.520 us.
FILE_FLAGS = {
    "awq_decode.hip": ["-mllvm", "-amdgpu-kernarg-preload-count=16"],
}


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = ([hipcc(), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj] + COMMON_FLAGS +
           FILE_FLAGS.get(src, []) + extra)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def build(verbose: bool = False, extra_flags: list[str] | None = None, jobs: int = 6) -> str:
    """Compile every HIP source for gfx950 and link the shared library, and
    where torch can be imported its Python module.  Always recompiles.
    Returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = list(extra_flags or [])
    try:
        import torch  # noqa: F401
        with_torch = True
    except ImportError:
        with_torch = False
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        bind = ex.submit(_compile_bind) if with_torch else None
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES + BENCH_SOURCES))
    _link(objs[:len(SOURCES)], LIB_PATH, verbose)
    _link(objs[len(SOURCES):], BENCH_LIB_PATH, verbose)
    if bind:
        _link_bind(bind.result(), verbose)
    elif verbose:
        print(f"{os.path.basename(BIND_PATH)} is left out: torch cannot be imported")
    return LIB_PATH


def _run(cmd: list[str], what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")


def _host_compiler(*language: str) -> list[str]:
    """g++, or the compiler that builds the library (given the language)."""
    gxx = shutil.which("g++")
    return [gxx] if gxx else [hipcc(), *language]


def _compile_bind() -> str:
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(BUILD_DIR, BIND_SOURCE + ".o")
    includes = [sysconfig.get_paths()["include"]] + cpp_extension.include_paths("cuda")
    _run(_host_compiler("-x", "c++") + ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
          "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}"] +
         [x for i in includes for x in ("-isystem", i)] +
         ["-c", os.path.join(CSRC, BIND_SOURCE), "-o", obj], f"compiling {BIND_SOURCE}")
    return obj


def _link_bind(obj: str, verbose: bool) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND_PATH + ".tmp"
    # torch has loaded its own libraries before it imports this one.
    _run(_host_compiler() + ["-shared", "-o", tmp, obj, f"-L{libs}", "-lc10", "-lc10_hip", "-ltorch_cpu",
          "-ltorch_python", f"-L{PKG_DIR}", f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"],
         "linking _serving.so")
    os.replace(tmp, BIND_PATH)
    if verbose:
        print(f"built {BIND_PATH}")


def _link(objs: list[str], path: str, verbose: bool) -> None:
    tmp = path + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, path)
    if verbose:
        print(f"built {path}")


if __name__ == "__main__":
    build(verbose=True, extra_flags=sys.argv[1:])
