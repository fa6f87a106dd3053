"""Build libsgemm_mi355.so in-tree with hipcc for gfx950.

Each HIP source compiles to an object in parallel, then one shared library is
linked next to this file. Device code is built with the packed-FP32 target
feature disabled, so the compiler emits only scalar FP32 vector arithmetic
(v_fma_f32 and friends) besides the FP32 matrix instructions.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libsgemm_mi355.so")
OBJDIR = os.path.join(ROOT, "_build")

SOURCES = ["kernels_mfma.hip", "kernels_mfma_dma.hip", "kernels_valu.hip", "kernels_util.hip", "sgemm_api.hip",
           "kernels_fp8_gemm.hip", "kernels_fp8_tile.hip", "kernels_fp8_skinny.hip",
           "kernels_fp8_quantize.hip", "kernels_route.hip", "kernels_norm.hip", "kernels_activation.hip",
           "kernels_experts.hip", "kernels_experts_tile.hip",
           "fp8_api.hip", "route_api.hip", "layer_api.hip", "experts_api.hip"]
ARCH = os.environ.get("SGEMM_MI355_ARCH", "gfx950")

HIPFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Werror",
    "-Wno-unused-command-line-argument",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str, extra=()) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *HIPFLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; that
    # warning is expected. Anything else is shown.
    noise = "not a recognized feature for this target"
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msg}")
    if msg.strip():
        print(msg, file=sys.stderr)
    return obj


def build(extra=()) -> str:
    """Compile every HIP source and link libsgemm_mi355.so; returns its path."""
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(sys.argv[1:]))
