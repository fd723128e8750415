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
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libfp8.so")
UNITS = [os.path.join(HERE, "csrc", f) for f in ("libfp8.cu", "passes.cu", "norm_bwd.cu")]
CALLS = os.path.join(HERE, "_calls.so")
CALLS_MAIN = os.path.join(HERE, "csrc", "calls.cpp")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu*"))) + [os.path.join(ROOT, "include", "fp8.h")]


def stale(lib: str, srcs: list[str]) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in srcs)


def _compile_units(verbose: bool) -> None:
    """The translation units side by side, then the library from them."""
    nvcc = os.environ.get("NVCC", "nvcc")
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, os.path.basename(u) + ".o") for u in UNITS]
        commands = [[nvcc, *NVCC_FLAGS, "-c", u, "-o", o] for u, o in zip(UNITS, objects)]
        if verbose:
            print("\n".join(" ".join(c) for c in commands), flush=True)
        running = [subprocess.Popen(c) for c in commands]
        codes = [r.wait() for r in running]
        for c, cmd in zip(codes, commands):
            if c:
                raise subprocess.CalledProcessError(c, cmd)
        _compile([nvcc, *NVCC_FLAGS, "-shared", *objects], LIB, verbose)


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
        _compile_units(verbose)
    if force or stale(CALLS, [CALLS_MAIN, os.path.join(ROOT, "include", "fp8.h")]):
        _compile(_calls_command(), CALLS, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
