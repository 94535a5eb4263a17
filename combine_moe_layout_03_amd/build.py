"""Build libmoe_ep.so in-tree with hipcc for gfx950.

Usage: python -m combine_moe_layout_03_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoe_ep.so")
SOURCES = ["capi.hip", "layout.hip", "fused.hip", "scatter.hip", "fp8.hip", "ranks.hip",
           "rank_fused.hip", "replica.hip",
           # the operators around the experts (moe_experts.h)
           "experts/experts.hip", "experts/gate.hip", "experts/combine_grad.hip",
           "experts/swiglu.hip", "experts/grouped_gemm.hip"]
# floor kernels for the benchmark (measurement only; not part of the C ABI)
FLOOR_LIB = os.path.join(PKG, "libmoe_floors.so")
FLOOR_SOURCES = ["floors.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-fvisibility=hidden",
    "-Wall",
    # packed f32 ops off: the compiler must not form v_pk_{add,mul,fma}_f32
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # leading scalar and pointer kernel arguments preloaded into registers at
    # launch (no round trip to the argument buffer before the first loads;
    # the combine measured 4.74 vs 4.83 us at 128 x 7168)
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
]


def _hipcc(out: str, sources, verbose: bool) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    srcs = [os.path.join(CSRC, s) for s in sources]
    tmp = out + ".tmp"
    cmd = [hipcc, *HIPCC_FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", "-o", tmp, *srcs]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed to build {os.path.basename(out)}")
    os.replace(tmp, out)
    return out


def build(verbose: bool = False) -> str:
    """libmoe_ep.so (the library) and libmoe_floors.so (the benchmark's floor
    kernels)."""
    _hipcc(FLOOR_LIB, FLOOR_SOURCES, verbose)
    return _hipcc(LIB, SOURCES, verbose)


if __name__ == "__main__":
    print(build(verbose=True))
