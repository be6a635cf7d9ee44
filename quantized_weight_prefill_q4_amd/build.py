"""Compile libmq.so for gfx950 in-tree with hipcc, and the torch binding of the
layer operators with the host compiler.

Usage: ``python -m quantized_weight_prefill_q4_amd.build`` (or ``build_lib()``).
Each ``csrc/*.hip`` file is compiled to an object under ``_build/`` in
parallel, then linked into ``quantized_weight_prefill_q4_amd/libmq.so``;
``csrc/binding*.cpp`` become the extension module ``_binding.so`` beside it.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libmq.so")
BINDING_PATH = os.path.join(PKG, "_binding.so")
SOURCES = ("mq_api.hip", "dequant.hip", "gemm.hip", "gemm_xf32.hip", "mmq.hip", "rms_norm.hip",
           "gemm_linear.hip", "gemm_glu.hip", "linear_rows.hip", "rope.hip", "kv_q4.hip",
           "attention_q4.hip", "attention_prompt.hip")

BINDING_SOURCES = ("binding.cpp", "binding_attention.cpp")

CXX = os.environ.get("CXX", shutil.which("g++") or "c++")
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


def _build_binding(verbose: bool) -> str:
    """csrc/binding*.cpp as a CPython extension against the installed torch."""
    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    inc = os.path.join(root, "include")
    tmp = BINDING_PATH + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           *(os.path.join(CSRC, s) for s in BINDING_SOURCES), "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def build_lib(verbose: bool = False) -> str:
    """Compile every HIP source and link libmq.so, and build the torch binding;
    returns the library path.  The library needs neither the host compiler nor
    Python's and torch's headers: it is linked also where the binding, which
    does, cannot be built, and that is raised afterwards."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if binding.exception() and os.path.exists(BINDING_PATH):
        os.remove(BINDING_PATH)   # an older library's
    binding.result()
    return LIB_PATH


if __name__ == "__main__":
    print(build_lib(verbose="-v" in sys.argv))
