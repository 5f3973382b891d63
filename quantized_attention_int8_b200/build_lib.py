"""Builds the CUDA library in-tree with nvcc for sm_100a: libsage_b200.so and its checked
twin libsage_b200_checked.so (-DSAGE_CHECKED: every kernel store tests its extent first); and
_sage_binding.<python>-torch<version>.so, the serving calls' Python binding (host code against torch's headers).

Usage: python quantized_attention_int8_b200/build_lib.py [--force] [--ptxas-info] [--no-checked] [--no-binding]

Without the binding the package has everything but the serving calls.

Run it as a script (not as a module of the package): importing the package
loads the library, which may not exist yet or may be stale.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsage_b200.so")
LIB_CHECKED = os.path.join(PKG, "libsage_b200_checked.so")
SOURCES = ["api.cu", "attn.cu", "quant.cu", "cache.cu", "decode.cu"]
HEADERS = ["sm100.cuh", "sage_internal.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsage_b200.so")
    return cand


def _stale(lib: str, sources: list[str]) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in sources] + [os.path.join(INCLUDE, "sage.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def _build_one(lib: str, defines: list[str], force: bool, ptxas_info: bool, verbose: bool) -> str:
    if not force and not _stale(lib, SOURCES + HEADERS):
        return lib
    tmp = lib + ".tmp"
    cmd = [_nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-shared",
           "--threads", "4", *defines, f"-I{INCLUDE}", f"-I{CSRC}", "-o", tmp,
           *[os.path.join(CSRC, f) for f in SOURCES]]
    if ptxas_info:
        cmd[1:1] = ["-Xptxas", "-v"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    if ptxas_info or verbose:
        sys.stderr.write(r.stdout + r.stderr)
    os.replace(tmp, lib)
    return lib


def _build_binding(force: bool, verbose: bool) -> None:
    import torch
    # named for the Python and the torch that it is built against: another one looks for a file of its own
    binding = os.path.join(PKG, f"_sage_binding.{sys.implementation.cache_tag}-torch{torch.__version__}.so")
    if not force and not _stale(binding, ["binding.cpp"]):
        return
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = binding + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           *[x for i in includes for x in ("-isystem", i)], "-o", tmp, os.path.join(CSRC, "binding.cpp"),
           f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, binding)


def build(force: bool = False, ptxas_info: bool = False, verbose: bool = False, checked: bool = True,
          binding: bool = True) -> str:
    """Builds the library (and, unless checked=False, its checked twin; unless binding=False, the serving calls'
    binding); returns the library's path."""
    _build_one(LIB, [], force, ptxas_info, verbose)
    if checked:
        _build_one(LIB_CHECKED, ["-DSAGE_CHECKED"], force, ptxas_info, verbose)
    if binding:
        _build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_info="--ptxas-info" in sys.argv, verbose=True,
          checked="--no-checked" not in sys.argv, binding="--no-binding" not in sys.argv)
