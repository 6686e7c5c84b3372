"""The library is built where the Python module beside it cannot be: without torch, or
without what compiles it."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from dense_fp16_gemm_05_gb300 import build as gbuild

WITHOUT_TORCH = """
import sys
class Block:
    def find_spec(self, name, path=None, target=None):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, Block())
from dense_fp16_gemm_05_gb300 import build
print(build.build())
assert "torch" not in sys.modules
"""


def test_the_library_needs_no_torch():
    gbuild.build()
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH], cwd=gbuild.ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[-1] == gbuild.LIB and "ctypes" in r.stderr


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A module's path of its own, and a library that is up to date."""
    gbuild.build()
    path = str(tmp_path / "_binding" / "_binding.so")
    monkeypatch.setattr(gbuild, "binding_path", lambda: path)
    return path


@pytest.mark.parametrize("compiler", ["false", "/nonexistent/c++"])
def test_the_library_needs_no_compiler_of_the_module(elsewhere, monkeypatch, capfd, compiler):
    monkeypatch.setenv("CXX", compiler)
    os.makedirs(os.path.dirname(elsewhere))
    with open(elsewhere, "wb") as f:
        f.write(b"of older sources")
    os.utime(elsewhere, (1, 1))
    assert gbuild.build() == gbuild.LIB
    assert "ctypes" in capfd.readouterr().err
    # what is older than its sources is not left for a library that it does not fit
    assert not os.path.exists(elsewhere)
    with pytest.raises((OSError, subprocess.CalledProcessError)):
        gbuild.build_binding()


def test_a_library_is_linked_where_the_module_fails(elsewhere, monkeypatch, tmp_path, capfd):
    """The whole way, with stand-ins for the compilers: every object is made and linked."""
    lib = str(tmp_path / "libgemm_f16.so")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho made > "$2"\n')
    nvcc.chmod(0o755)
    monkeypatch.setattr(gbuild, "LIB", lib)
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setenv("CXX", "false")
    assert gbuild.build() == lib and os.path.exists(lib)
    assert "ctypes" in capfd.readouterr().err
