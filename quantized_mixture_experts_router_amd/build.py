"""Build libqmoe.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree.

Usage: python -m quantized_mixture_experts_router_amd.build [--jobs N]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqmoe.so")

SOURCES = [
    "qmoe_plan.cpp",
    "qmoe_api.cpp",
    "qmoe_gmm.cpp",
    "qmoe_moe.cpp",
    "qmoe_tokens.cpp",
    "qmoe_linear.cpp",
    "qmoe_rows8.cpp",
    "qmoe_norm.cpp",
    "qmoe_route_scored.cpp",
    "kernels/route.hip",
    "kernels/operand.hip",
    "kernels/gemm.hip",
    "kernels/stream.hip",
    "kernels/stream_half.hip",
    "kernels/tiled.hip",
    "kernels/gmm.hip",
    "kernels/gmm_typed.hip",
    "kernels/moe.hip",
    "kernels/tokens.hip",
    "kernels/rows8.hip",
    "kernels/norm.hip",
    "kernels/route_scored.hip",
    "kernels/linear_ops.hip",
    "kernels/linear_f16.hip",
    "kernels/linear_bf16.hip",
    "kernels/linear_f32.hip",
]

ARCH = os.environ.get("QMOE_OFFLOAD_ARCH", "gfx950")

CFLAGS = [
    "-O3", "-fPIC", "-std=c++17", f"--offload-arch={ARCH}",
    # packed fp32 VALU forms stay off: plain fp32 arithmetic only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
] + [f for f in os.environ.get("QMOE_EXTRA_CFLAGS", "").split() if f]


def _hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src.replace("/", "_") + ".o")
    cmd = [_hipcc(), *CFLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def build(jobs: int | None = None, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(8, len(SOURCES))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=None)
    a = ap.parse_args()
    build(a.jobs, verbose=True)
    sys.exit(0)
