"""Builds libq4gemv.so in-tree with nvcc for sm_100a (no torch extension
machinery: the library is a plain C-ABI shared object)."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libq4gemv.so")
SOURCES = ["q4gemv_api.cu", "q4gemv_noalloc.cu", "mix_api.cu"]
HEADERS = ["device_common.cuh", "partition.cuh", "gemv_dp2a.cuh", "gemv_mma.cuh", "stack.cuh",
           "gemm_tc.cuh", "gemv_swiglu.cuh", "gemv_tcs.cuh", "ctx_view.h", "mix_common.cuh",
           "kv_append.cuh", "attn_rows.cuh", "attn_split.cuh", "mma_common.cuh",
           "lin_chunk.cuh", "attn_tc.cuh", "tc_common.cuh", "lin_seg.cuh",
           "lin_tc.cuh", "linattn.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(os.path.dirname(HERE), "include", "q4gemv.h"))
    return files


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-rdc=false",
           "-Xcompiler", "-fvisibility=hidden", "-cudart", "static",
           "-o", tmp, *[os.path.join(CSRC, f) for f in SOURCES]]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.check_call(cmd, cwd=CSRC)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
