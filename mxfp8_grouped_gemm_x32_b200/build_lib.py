"""Builds libmoe_mxfp8.so (the C-ABI CUDA library) in-tree for sm_100a.

    python -m mxfp8_grouped_gemm_x32_b200.build_lib [--force]
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmoe_mxfp8.so")
SOURCES = ["moe_mxfp8_all.cu", "api.cu", "gemm.cu", "permute.cu", "quant.cu", "swiglu_bwd.cu", "noalloc.cu", "router.cu",
           "scales.cu", "transpose.cu", "common.cuh", "gemm.cuh", "permute.cuh", "quant.cuh", "swiglu_bwd.cuh",
           "router.cuh", "scales.cuh", "transpose.cuh", "router_loss.cu", "router_loss.cuh", "mxfp4.cu", "mxfp4.cuh",
           "gemm_mxfp4.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "-diag-suppress", "550"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "include", "moe_mxfp8.h")]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    cmd = [_nvcc(), *NVCC_FLAGS, "-o", LIB + ".tmp", os.path.join(CSRC, "moe_mxfp8_all.cu")]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
