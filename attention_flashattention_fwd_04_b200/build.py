"""Compile the CUDA library (sm_100a) into the package directory.

``python -m attention_flashattention_fwd_04_b200.build`` or ``build()``.  The
results, ``libattn_b200.so`` and ``_attn_torch.so`` (argument marshalling of the
8-bit cache's calls, against PyTorch's headers), sit next to this file and are
what :mod:`.api` loads.  nvcc cross-compiles, so no GPU is needed to build.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libattn_b200.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
TORCH_PATH = os.path.join(PKG_DIR, "_attn_torch.so")
TORCH_SOURCE = os.path.join(CSRC, "attn_torch.cpp")
HEADER = os.path.join(INCLUDE, "attn_b200.h")
SOURCES = ["attn_lib.cu", "attn_noalloc.cu"]  # attn_lib.cu includes attn_api.cu

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build the library")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))]
    files.append(os.path.join(INCLUDE, "attn_b200.h"))
    return files


def _newer(target, inputs) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB_PATH, _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Build ``libattn_b200.so`` and ``_attn_torch.so`` unless they are newer
    than every source."""
    build_torch(force, verbose)
    if not force and up_to_date():
        return LIB_PATH
    tmp = LIB_PATH + ".tmp"
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-o", tmp, *(os.path.join(CSRC, s) for s in SOURCES)]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build_torch(force: bool = False, verbose: bool = False) -> str:
    """Build ``_attn_torch.so`` (host code only: the C++ compiler) unless it is
    newer than its sources."""
    if not force and _newer(TORCH_PATH, [TORCH_SOURCE, HEADER]):
        return TORCH_PATH
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = TORCH_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           *(f"-isystem{d}" for d in [*include_paths("cuda"), sysconfig.get_paths()["include"]]), TORCH_SOURCE, "-o", tmp,
           *(f"-L{d}" for d in library_paths()), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, TORCH_PATH)
    return TORCH_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
