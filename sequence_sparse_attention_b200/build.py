"""Build libspava.so (sm_100a, nvcc) and _calls.so (its compiled PyTorch calls, g++) in-tree.

    python -m sequence_sparse_attention_b200.build [--verbose]

The library is self-contained: the CUDA runtime is linked statically and the
driver entry point for TMA descriptors is resolved at run time, so the .so
loads on a machine without a GPU (its calls then report SPAVA_ERR_CUDA).
_calls.so is a Python extension module that links it and torch.
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
LIB = os.path.join(PKG, "libspava.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "calls.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("spava_api.cu", "cache_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
    os.path.join(ROOT, "include", "spava.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "static",
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def stale(target: str, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in deps)


def compile_to(target: str, cmd) -> None:
    tmp = target + f".tmp{os.getpid()}"
    subprocess.check_call([*cmd, "-o", tmp])
    os.replace(tmp, target)


def build_calls() -> None:
    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    compile_to(CALLS, [
        "g++", "-O2", "-std=c++17", "-fPIC", "-shared", *("-I" + d for d in include),
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", CALLS_SOURCE, LIB,
        "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
        "-Wl,-rpath,$ORIGIN"])


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale(LIB, DEPS):
        # the soname lets _calls.so find the library beside it
        compile_to(LIB, [nvcc(), *NVCC_FLAGS, "-Xlinker", "-soname=libspava.so",
                         *(["-Xptxas", "-v"] if verbose else []), *SOURCES])
    if force or stale(CALLS, [CALLS_SOURCE, os.path.join(ROOT, "include", "spava.h")]):
        build_calls()
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
