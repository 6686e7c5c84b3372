"""Builds the CUDA library ``libgemm_f16.so`` in-tree with nvcc for sm_103a.

Translation units: ``csrc/gemm_f16.cu`` (the C ABI) and ``csrc/gemm_cfg_<id>.cu``
(the kernel instances of each configuration), compiled in parallel with one
``-gencode`` (``arch=compute_103a,code=sm_103a``) and linked with the CUDA
runtime linked statically, so the library loads on machines without a GPU
driver (the symbol-export test runs there).  Beside it ``csrc/binding.cpp``, a
Python module on the C++ side of torch, is compiled with the host compiler; the
library needs neither it nor torch, and is made where the module cannot be.  What is
newer than its sources is not built again (the module: and was built for this torch).
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgemm_f16.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
    "-cudart", "static",
]


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.inc")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def binding_path() -> str:
    """The module of csrc/binding.cpp, which knows the tensors of one torch alone."""
    import torch
    return os.path.join(PKG, "_binding", torch.__version__.replace("+", "_"), "_binding.so")


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compiles csrc/binding.cpp for this torch if it is missing or stale; returns the module's path."""
    import sysconfig

    import torch
    out = binding_path()
    headers = glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(out):
        t = os.path.getmtime(out)
        if all(os.path.getmtime(s) <= t for s in (BINDING_SOURCE, *headers)):
            return out
    os.makedirs(os.path.dirname(out), exist_ok=True)
    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda", "include")
    tmp = out + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f'-DBINDING_TORCH_VERSION="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", os.path.join(base, "include"), "-I", cuda, "-I", sysconfig.get_paths()["include"],
           "-o", tmp, BINDING_SOURCE, "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python", "-ltorch"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    try:
        subprocess.run(cmd, check=True)
    except (OSError, subprocess.CalledProcessError):
        if os.path.exists(out):   # of older sources: none is better
            os.unlink(out)
        raise
    os.replace(tmp, out)
    return out


def _try_binding(force: bool = False, verbose: bool = False) -> None:
    """build_binding, or a line that says why not: the module only shortens calls."""
    try:
        build_binding(force, verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        print(f"csrc/binding.cpp is not built, calls go through ctypes: {e}", file=sys.stderr)


def _translation_units() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compiles the library, and where it can the Python module, if they are missing or stale; returns the library's path.

    Each translation unit (the C ABI and one per kernel configuration) is
    compiled to an object in parallel, then the objects are linked into one
    shared library.
    """
    import concurrent.futures
    import tempfile
    if not force and os.path.exists(LIB):
        lib_t = os.path.getmtime(LIB)
        if all(os.path.getmtime(s) <= lib_t for s in _sources()):
            _try_binding(verbose=verbose)
            return LIB
    tmpdir = tempfile.mkdtemp(prefix="gemm_f16_build")
    compile_flags = [f for f in NVCC_FLAGS if f not in ("-shared", "-cudart", "static")]
    units = _translation_units()

    def compile_one(src):
        obj = os.path.join(tmpdir, os.path.basename(src) + ".o")
        cmd = [nvcc(), *compile_flags, *(extra_flags or []), "-I", INCLUDE, "-c", "-o", obj, src]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(units) + 1, os.cpu_count() or 4)) as ex:
        module = ex.submit(_try_binding, force, verbose)
        objs = list(ex.map(compile_one, units))
    tmp = LIB + f".tmp{os.getpid()}"
    link = [nvcc(), "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-cudart", "static", "-o", tmp, *objs]
    if verbose:
        print(" ".join(link), file=sys.stderr)
    subprocess.run(link, check=True)
    os.replace(tmp, LIB)
    for o in objs:
        os.unlink(o)
    os.rmdir(tmpdir)
    module.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
