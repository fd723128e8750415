"""Build libfp8.so (all CUDA kernels, sm_100a) in-tree with nvcc, and _calls.so
(the short way from tensors to its block-scaled operators) with g++.

    python -m fp8_mixed_precision_tensor_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libfp8.so")
MAIN = os.path.join(HERE, "csrc", "libfp8.cu")
CALLS = os.path.join(HERE, "_calls.so")
CALLS_MAIN = os.path.join(HERE, "csrc", "calls.cpp")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-shared",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu*"))) + [os.path.join(ROOT, "include", "fp8.h")]


def stale(lib: str, srcs: list[str]) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in srcs)


def _compile(cmd: list[str], lib: str, verbose: bool) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [*cmd, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, lib)


def _calls_command() -> list[str]:
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(os.environ.get("NVCC", "nvcc")))))
    includes = [*ext.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    libs = ext.library_paths()
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f'-DFP8_TORCH_VERSION="{torch.__version__}"', *(a for d in includes for a in ("-isystem", d)), CALLS_MAIN,
            *(f"-L{d}" for d in libs), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale(LIB, sources()):
        _compile([os.environ.get("NVCC", "nvcc"), *NVCC_FLAGS, MAIN], LIB, verbose)
    if force or stale(CALLS, [CALLS_MAIN, os.path.join(ROOT, "include", "fp8.h")]):
        _compile(_calls_command(), CALLS, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
