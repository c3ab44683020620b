"""Build step of libsa2: compiles every CUDA source under csrc/ for sm_103a with nvcc (one
process per translation unit, in parallel) and links the in-tree shared library
``libsa2.so`` next to this file, then the extension module ``_cross`` (csrc/cross_binding.cpp, with
the host compiler and torch's headers), which is linked to it.  Objects go to ``_build/``.  A host without
torch, which has the C ABI alone, gets ``libsa2.so`` alone.

Usage: python -m block_sparse_attention_sa2_gb300.build_lib [--force] [--verbose]
(without torch: python block_sparse_attention_sa2_gb300/build_lib.py)
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsa2.so")
BINDING = os.path.join(PKG, "_cross.so")
BINDING_FOR = os.path.join(BUILD, "_cross.for")  # what _cross.so was built for
BINDING_SRC = os.path.join(CSRC, "cross_binding.cpp")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                 "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def _torch():
    """torch, or None on a host without it."""
    try:
        import torch
    except ImportError:
        return None
    return torch


def _binding_for(torch) -> str:
    """The Python and torch that a binding built now is for."""
    return f"{sys.implementation.cache_tag} torch {torch.__version__} {torch.__file__}"


def _newer(target: str, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def up_to_date() -> bool:
    """Whether libsa2.so, and with torch its binding for that torch, are newer than their sources."""
    if not _newer(LIB, _sources() + _headers()):
        return False
    torch = _torch()
    if torch is None:
        return True
    if not _newer(BINDING, [BINDING_SRC] + _headers()) or not os.path.exists(BINDING_FOR):
        return False
    with open(BINDING_FOR) as f:
        return f.read() == _binding_for(torch)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + CFLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    log = os.path.join(BUILD, os.path.basename(src)[:-3] + ".log")
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stdout.write(r.stderr)
    return obj


def _compile_binding(torch) -> str:
    import sysconfig
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    obj = os.path.join(BUILD, "cross_binding.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", inc,
           "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda, "-I", sysconfig.get_paths()["include"],
           "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str, torch) -> None:
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-lsa2", "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(_binding_for(torch))


def _link_library(objs) -> None:
    tmp = LIB + ".tmp"
    # static CUDA runtime; driver entry points are resolved at run time, so no -lcuda
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libsa2.so, then with torch its binding (skipped when they are newer than every source).
    A binding that fails to build raises, after libsa2.so has been linked."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs, torch = _sources(), _torch()
    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = None if torch is None else ex.submit(_compile_binding, torch)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    _link_library(objs)
    if binding is None:
        print("build_lib: no torch on this host: libsa2.so alone, without the Python binding _cross.so", file=sys.stderr)
    else:
        _link_binding(binding.result(), torch)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
