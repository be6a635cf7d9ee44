"""Compile libmq.so for gfx950 in-tree with hipcc.

Usage: ``python -m quantized_weight_prefill_q4_amd.build`` (or ``build_lib()``).
Each ``csrc/*.hip`` file is compiled to an object under ``_build/`` in
parallel, then linked into ``quantized_weight_prefill_q4_amd/libmq.so``.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libmq.so")
SOURCES = ("mq_api.hip", "dequant.hip", "gemm.hip", "gemm_xf32.hip", "mmq.hip", "rms_norm.hip",
           "gemm_linear.hip", "gemm_glu.hip", "linear_rows.hip")

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")

# Device code: gfx950 only; keep IEEE denormals (f16 subnormal weights must
# survive the decode); no implicit contraction (the decode's roundings are
# written out explicitly); packed-f32 VALU forms disabled.
CFLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fno-gpu-flush-denormals-to-zero",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
    "-I", INCLUDE,
    "-I", CSRC,
]


# Per-file additions.  MFMA results in VGPRs, where the VALU reads them (instead
# of AGPR copies): mmq.hip scales each block's integer dot, linear_rows.hip has
# few accumulators.
_VGPR_FORM = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
EXTRA = {"mmq.hip": _VGPR_FORM, "linear_rows.hip": _VGPR_FORM}


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build_lib(verbose: bool = False) -> str:
    """Compile every HIP source and link libmq.so; returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build_lib(verbose="-v" in sys.argv))
