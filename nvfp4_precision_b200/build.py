"""Build the CUDA library ``libfp4attn.so`` in-tree for sm_100a, and the
extension through which Python makes its shortest calls.

    python -m nvfp4_precision_b200.build [--force] [--verbose]

Plain nvcc, one shared library, static CUDA runtime; the C ABI is declared in
include/fp4attn.h at the repository root.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfp4attn.so")
# The same library with every kernel's global stores, atomics and tile
# coordinates checked against their buffers (-DFP4ATTN_BOUNDS_CHECK): a failed
# check records FP4ATTN_ERR_RANGE instead of touching memory.  A debugging
# build; the binding loads it when FP4ATTN_BOUNDS_CHECK=1.
LIB_CHECKED = os.path.join(PKG, "libfp4attn_checked.so")

CALLS_SRC = os.path.join(CSRC, "calls.cpp")


def calls_path() -> str:
    """The extension with the calls of the linear layers and norms from Python
    (csrc/calls.cpp).  It holds for one Python and one torch, which its name
    tells: after a change of either it is not there until it is built again."""
    import torch
    return os.path.join(PKG, f"_calls.{sys.implementation.cache_tag}.torch-{torch.__version__}.so")


NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-shared", "--threads", "0",  # sources in parallel
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def build_calls(force: bool = False) -> str:
    out = calls_path()
    deps = [CALLS_SRC, os.path.join(INCLUDE, "fp4attn.h")]
    if not force and os.path.exists(out) and all(os.path.getmtime(out) >= os.path.getmtime(d) for d in deps):
        return out
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = out + f".tmp{os.getpid()}"
    includes = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in includes),
                    CALLS_SRC, f"-L{root}/lib", f"-Wl,-rpath,{root}/lib", "-ltorch_python", "-ltorch", "-ltorch_cpu",
                    "-lc10", "-lc10_cuda", "-o", tmp], check=True)
    os.replace(tmp, out)
    return out


def build_library(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    out = LIB_CHECKED if checked else LIB
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(out) and all(os.path.getmtime(out) >= os.path.getmtime(d) for d in deps):
        return out
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC]
    if checked:
        cmd += ["-DFP4ATTN_BOUNDS_CHECK"]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += [*sources(), "-o", tmp]
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    # the library first: the attention does not need the extension
    out = build_library(force, verbose, checked)
    build_calls(force and not checked)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv, checked="--checked" in sys.argv))
