"""Build the in-tree CUDA library ``libwush.so`` for sm_100a with nvcc.

Usage: ``python -m blockwise_adaptive_transforms_b200._build [--force] [--verbose]``.
The library is rebuilt when any source under csrc/ or include/ is newer than it.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
LIB_PATH = os.path.join(PKG_DIR, "libwush.so")
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _sources():
    return sorted(glob.glob(os.path.join(PKG_DIR, "csrc", "*.cu")) +
                  glob.glob(os.path.join(PKG_DIR, "csrc", "*.cuh")) +
                  glob.glob(os.path.join(PKG_DIR, "csrc", "*.h")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libwush.so")


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu into libwush.so next to this file and return its path."""
    if not force and not needs_build():
        return LIB_PATH
    units = sorted(glob.glob(os.path.join(PKG_DIR, "csrc", "*.cu")))
    tmp = LIB_PATH + ".tmp"
    cmd = [_nvcc(), "-O3", "-std=c++17", *ARCH_FLAGS, "-lineinfo", "-Xcompiler", "-fPIC",
           "-shared", "--threads", "0", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG_DIR, "csrc"),
           "-o", tmp, *units]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
