"""Compiles the CUDA library ``libk3da.so`` in-tree for sm_103a.

Usage: ``python -m speculative_decoding_drafter_k3_gb300.build`` (or through
``__graft_entry__.build()``).  nvcc cross-compiles on a machine without a GPU.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", f) for f in
           ("k3da.cu", "k3da_norm_rope.cu", "k3da_cache.cu", "k3da_chunk.cu", "k3da_chunk_small.cu")]
HEADERS = [os.path.join(ROOT, "include", "k3da.h")] + [os.path.join(PKG, "csrc", f) for f in
           ("rope_table.h", "cache_common.cuh", "chunk_cut.h", "chunk_plan.cuh", "sm103.cuh", "tensor_maps.h")]
LIB = os.path.join(PKG, "libk3da.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libk3da.so")
    return cand


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in SOURCES + HEADERS)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--threads", "0", "-Xcompiler", "-fPIC",
           "-shared", "-I", os.path.join(ROOT, "include"), "-o", tmp, *SOURCES,
           "-cudart", "static", *extra]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
