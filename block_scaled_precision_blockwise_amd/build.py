"""Builds libbsq.so (the HIP kernels and the C ABI) in-tree for gfx950.

    python -m block_scaled_precision_blockwise_amd.build

Every HIP translation unit is compiled with hipcc for gfx950 only, with
packed-FP32 instruction selection disabled, and linked into
block_scaled_precision_blockwise_amd/libbsq.so next to this file.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbsq.so")
SOURCES = ["api.hip", "api_moe.hip", "quant.hip", "gemm.hip", "route.hip", "rows.hip", "gate.hip", "moe_gemm.hip",
           "api_mx4.hip", "quant4.hip", "gemm4.hip", "norm.hip"]
HEADERS = ["common.h", "fp4.h", "fp8.h", "lds.h", "quant.h", "quant4.h", "gemm.h", "gemm4.h", "moe.h",
           "moe_index.h", "mx4_index.h", "norm.h", "tiles.h"]

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")

CFLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-result",
    "-I" + INCLUDE,
    "-I" + CSRC,
    # no packed FP32 (v_pk_*_f32) instruction selection
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr[-6000:]}")
    return obj


def build(verbose: bool = False) -> str:
    """Compile and link; returns the path of libbsq.so."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-6000:]}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
