"""Build libdynconv.so for gfx950 with hipcc, in-tree.

    python -m input_dependent_depthwise_amd.build

compiles every ``csrc/*.hip`` into ``_build/`` and links
``input_dependent_depthwise_amd/libdynconv.so``.  hipcc cross-compiles, so
this works on a machine without a GPU.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdynconv.so")
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Werror",
    "-Wno-unused-function", "-I", INCLUDE, "-I", CSRC,
    # keep the compiler from emitting packed fp32 VALU ops (v_pk_fma_f32 and kin)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]
# Per-file additions.  The low-rank forward consumes each matrix-core result
# on the VALU once: with the results in VGPRs (this target's MFMAs write them
# directly) it needs no v_accvgpr_read copy per element.  Kernels that keep
# accumulating in the matrix cores are better off with AGPR accumulators.
FILE_FLAGS = {
    "conv_fwd_lowrank.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    # one wave per SIMD holds more than 256 registers here: without it every score block is copied
    # between the two halves of the register file
    "attn_bwd_bf16.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "attn_window_bwd_bf16.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *CFLAGS, *FILE_FLAGS.get(os.path.basename(src), []), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; that line is harmless
    noise = "'-packed-fp32-ops' is not a recognized feature"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def build(jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    jobs = jobs or min(len(srcs), max(1, (os.cpu_count() or 4)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
