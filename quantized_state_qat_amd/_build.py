"""Build liblaqat.so (the HIP kernels and the C ABI) in-tree with hipcc for gfx950."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblaqat.so")
SOURCES = ["la_api.cpp", "fwd.hip", "fwd_fast.hip", "fwd_wave.hip", "fwd_mfma.hip", "fwd_tok.hip", "decode.hip", "bwd.hip",
           "bwd_mfma.hip", "noalloc.hip", "chunk_fwd.hip", "chunk_bwd.hip", "la_layer.cpp", "layer_conv.hip", "layer_norm.hip",
           "scan_step.hip", "scan_fwd.hip", "scan_bwd.hip", "la_proj.cpp", "linear_fwd.hip", "linear_bwd.hip", "gate_norm.hip", "gate_bwd.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "-std=c++20", "-O3", "-fPIC", "--offload-arch=gfx950",
    # contraction only where the source writes fmaf: the forward and the backward's recompute
    # must round identically
    "-ffp-contract=off",
    # no packed FP32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # matrix-core results in ordinary VGPRs (gfx950 allows it): no accumulator-register copies
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",
    "-Wall", "-Wno-unused-function",
]
# The products' tiles: accumulators in the accumulator registers, which leaves the others to the operands.
WITHOUT = {"linear_fwd.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"], "linear_bwd.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def _flags(src: str) -> list:
    drop = WITHOUT.get(src, [])
    at = next((i for i in range(len(FLAGS)) if drop and FLAGS[i:i + len(drop)] == drop), len(FLAGS))
    return FLAGS[:at] + FLAGS[at + len(drop):]


def _compile(src: str) -> str:
    obj = os.path.join(OUT, src + ".o")
    cmd = [HIPCC, *_flags(src), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    """Compile every source and link liblaqat.so.  Always recompiles."""
    os.makedirs(OUT, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
