"""Build libedit_attn.so in-tree with nvcc for sm_100a (cross-compiles without a GPU)."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", f) for f in ("edit_attn.cu", "edit_noalloc.cu", "packed_ops.cu")]
OUT = os.path.join(PKG, "libedit_attn.so")
DEPS = [os.path.join(PKG, "csrc", f) for f in ("edit_attn.cu", "edit_noalloc.cu", "common.cuh", "tc_gemm.cuh",
                                                "tc_conv.cuh", "simt_kernels.cuh", "sdpa_tc.cuh", "packed_ops.cu",
                                                "host.h", "packed_seq.cuh", "packed_attn.cuh", "packed_attn_tc.cuh", "delta_rule.cuh", "delta_chunk.cuh",
                                                "block_norm.cuh")]
DEPS.append(os.path.join(ROOT, "include", "edit_attn.h"))

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "-diag-suppress", "177", "--threads", "0"]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def up_to_date():
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(d) <= t for d in DEPS if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return OUT
    tmp = OUT + ".tmp"
    cmd = [nvcc(), *NVCC_FLAGS, "-o", tmp, *SRCS]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
