"""Build libtwotower.so in-tree with nvcc for sm_100a.

Usage: python -m block_wise_diffusion_b200.build [--force]
The library links the CUDA runtime statically, so it loads in processes
without a GPU (for symbol checks); every compute call needs a B200.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtwotower.so")
SOURCES = ["tt_api.cu", "tt_gemm.cu", "tt_attn.cu", "tt_small.cu", "tt_noalloc.cu",
           "tt_api_q8.cu", "tt_attn_q8.cu", "tt_attn_q8_rows.cu", "tt_cache_q8.cu", "tt_gemm_i8.cu"]
HEADERS = ["tt_internal.h", "tt_ptx.cuh", "tt_q8.h", "tt_quant.cuh", "tt_attn_q8.cuh",
           os.path.join("..", "..", "include", "twotower.h")]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared", "-cudart", "static", "--threads", "0",
    "-Xptxas", "-warn-spills",
]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [NVCC, *FLAGS, "-o", tmp, *[os.path.join(CSRC, s) for s in SOURCES]]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, flush=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
