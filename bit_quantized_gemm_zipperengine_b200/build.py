"""Build libmosaic.so (CUDA, sm_100a) in-tree with nvcc, and the _marshal extension (the operators'
operand checks, C++ against PyTorch's headers) with g++."""
from __future__ import annotations

import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmosaic.so")
# the same library with MQ_TIMELINE defined: the small decode GEMM records per-CTA event
# times (mq_timeline_read); used by timeline.py, never by the path
LIB_TIMELINE = os.path.join(PKG, "libmosaic_timeline.so")

MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")


def marshal_path() -> str:
    """The extension for the running interpreter and its PyTorch, which its name states: one built
    for others is never loaded."""
    return os.path.join(PKG, f"_marshal.{sys.implementation.cache_tag}-torch{importlib.metadata.version('torch')}.so")


NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    # IEEE fp32 division / rounding are part of the quantization spec: no fast math,
    # no contraction of multiply-add pairs.
    "-fmad=false", "-prec-div=true", "-prec-sqrt=true", "-ftz=false",
    "-Xcompiler", "-fPIC", "-shared",
    "-I" + INCLUDE, "-I" + CSRC,
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return (sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(INCLUDE, "*.h")))
            + [__file__])


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in deps())


def build(force: bool = False, verbose: bool = False, timeline: bool = False) -> str:
    """The C library, then (but not for the timeline's) the extension. The library needs nvcc alone:
    it is there, and up to date, when the extension cannot be built."""
    lib = build_lib(force, verbose, timeline)
    if not timeline:
        build_marshal(force)
    return lib


def build_lib(force: bool = False, verbose: bool = False, timeline: bool = False) -> str:
    lib = LIB_TIMELINE if timeline else LIB
    if not (force or stale(lib)):
        return lib
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, *(["-DMQ_TIMELINE"] if timeline else []), *(["-Xptxas", "-v"] if verbose else []),
           "-o", tmp, *sources()]
    subprocess.check_call(cmd)
    os.replace(tmp, lib)
    return lib


def build_marshal(force: bool = False) -> str:
    """The Python extension, built for the running interpreter and its PyTorch."""
    out = marshal_path()
    newest = max(os.path.getmtime(p) for p in [MARSHAL_SRC, __file__, *glob.glob(os.path.join(INCLUDE, "*.h"))])
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(os.environ.get("NVCC", "nvcc")) or "/usr/local/cuda/bin/nvcc")))
    tmp = out + f".tmp{os.getpid()}"
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
        "-isystem", os.path.join(base, "include"), "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
        "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"], "-o", tmp, MARSHAL_SRC,
        "-L" + os.path.join(base, "lib"), "-Wl,-rpath," + os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_python"])
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    build_lib(force=True, verbose="-v" in sys.argv)
    print(LIB)
    if "--lib" not in sys.argv:  # the C library alone
        print(build_marshal(force=True))
