"""The build where torch or g++ is missing."""
import os
import subprocess
import sys
import textwrap

import pytest

from bit_weight_quantized_awq_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_is_built_without_torch(tmp_path):
    """The C library needs hipcc alone; without torch there is nothing that
    its Python module could be for."""
    program = textwrap.dedent("""
        import importlib.util, sys
        sys.modules["torch"] = None          # import torch raises
        spec = importlib.util.spec_from_file_location("build", sys.argv[1])
        build = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(build)
        linked = []
        build.BUILD_DIR = sys.argv[2]
        build._compile = lambda src, extra: src + ".o"
        build._link = lambda objs, path, verbose: linked.append(path)
        assert build.build(verbose=True) == build.LIB_PATH
        assert linked == [build.LIB_PATH, build.BENCH_LIB_PATH]
        """)
    res = subprocess.run([sys.executable, "-c", program, build.__file__, str(tmp_path)],
                         capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr
    assert "torch" in res.stdout      # says what was left out


def test_python_module_is_built_without_gxx(tmp_path, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("HIPCC", build.hipcc())
    monkeypatch.setenv("PATH", "/nowhere")
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "BIND_PATH", str(tmp_path / "_serving.so"))
    build._link_bind(build._compile_bind(), False)
    assert os.path.getsize(tmp_path / "_serving.so") > 0
