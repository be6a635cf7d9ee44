"""Torch front end of the operators around the quantized products: linear layers
(the product with bias, activation and residual in its epilogue), gated pairs of
them, and the residual RMS norm that feeds them.

As in ``api``, every step of the computation runs in the HIP library.  A layer's
arguments are checked, its outputs allocated and the library called by one
native function (``csrc/binding.cpp``), on the current stream of the tensors'
device.  All tensors of a call must be on one GPU; it need not be the current
one.  Results are not recorded by autograd: the weights are fixed after load and
the operators have no backward pass.
"""

from __future__ import annotations

import ctypes
import functools
import importlib
import os

import torch

from ._lib import MQ_F16, MQ_F32, check, lib
from .api import _as_int, _fmt

_TYPES = {torch.float32: MQ_F32, torch.float16: MQ_F16}

# activations of a linear layer (include/mq.h)
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")
_ENTRY_POINTS = ("mq_linear_workspace_bytes", "mq_glu_workspace_bytes", "mq_linear_f16cache",
                 "mq_linear_fused", "mq_glu_f16cache", "mq_glu_fused", "mq_add_rms_norm",
                 "mq_add_rms_norm_q8_1", "mq_row_bytes", "mq_rope", "mq_kv_store_q4",
                 "mq_kv_load_q4", "mq_attention_q4", "mq_attention_q4_workspace_bytes")

_raw_stream = torch._C._cuda_getCurrentRawStream if torch.version.hip else None
_current_device = torch._C._cuda_getDevice if torch.version.hip else None


@functools.lru_cache(maxsize=None)
def _binding():
    """The native binding with libmq's entry points (loaded once).  Raises if
    either has not been built."""
    handle = lib()
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is missing: build it with "
                           "`python -m quantized_weight_prefill_q4_amd.build`")
    module = importlib.import_module("._binding", __package__)
    module.bind({n: ctypes.cast(getattr(handle, n), ctypes.c_void_p).value
                 for n in _ENTRY_POINTS})
    return module


def _on_device(x, call, where: str, args):
    """call(stream, *args) on the current stream of x's GPU, with that GPU
    current; a library status it returns is raised."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    dev = x.get_device()
    if dev == _current_device():
        r = call(_raw_stream(dev), *args)
    else:
        with torch.cuda.device(dev):
            r = call(_raw_stream(dev), *args)
    if r.__class__ is int:
        check(r, where)
    return r


def _act(act) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}: one of {list(ACTIVATIONS)}")
    return code


def _out_type(dtype) -> int:
    code = _TYPES.get(dtype)
    if code is None:
        raise ValueError(f"out_dtype must be float32 or float16, got {dtype}")
    return code


def linear_workspace_bytes(fmt, M: int, N: int, K: int, split_k: int = 0, x_f32: bool = False,
                           glu: bool = False) -> int:
    """Workspace bytes of a linear layer (fmt 0 / "f16": the f16 cache), or with
    ``glu`` of a gated one with N output columns; x_f32 for f32 activations."""
    f = 0 if fmt in (0, None, "f16") else _fmt(fmt)
    name = "mq_glu_workspace_bytes" if glu else "mq_linear_workspace_bytes"
    return check(getattr(lib(), name)(f, MQ_F32 if x_f32 else MQ_F16, _as_int(M), _as_int(N),
                                      _as_int(K), _as_int(split_k)), name)


def linear_f16cache(x: torch.Tensor, w16: torch.Tensor, K: int | None = None,
                    bias: torch.Tensor | None = None, act: str | None = None,
                    residual: torch.Tensor | None = None,
                    out_dtype: torch.dtype = torch.float32, split_k: int = 0,
                    out: torch.Tensor | None = None,
                    ws: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = act(x[:, :K] @ w16[:, :K]^T + bias) + residual, in out_dtype
    (f32 or f16): gemm_f16cache with the layer's epilogue.

    x [M, >=K] f16 (or f32, rounded to f16), w16 the f16 cache [N, ld], bias
    f32 [N], act one of ACTIVATIONS, residual [M, N] f32 or f16.  With out, y is
    of its type; out may be the residual itself (the stream is then updated in
    place)."""
    return _on_device(x, _binding().layer, "mq_linear_f16cache",
                      (x, w16, 0, -1, K, bias, _act(act), residual, False,
                       _out_type(out_dtype), split_k, out, ws))


def linear_fused(x: torch.Tensor, wq: torch.Tensor, fmt, N: int, K: int | None = None,
                 bias: torch.Tensor | None = None, act: str | None = None,
                 residual: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                 split_k: int = 0, out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None) -> torch.Tensor:
    """linear_f16cache straight from the quantized weight wq [N rows of K]."""
    return _on_device(x, _binding().layer, "mq_linear_fused",
                      (x, wq, _fmt(fmt) or -1, N, K, bias, _act(act),
                       residual, False, _out_type(out_dtype), split_k, out, ws))


def glu_f16cache(x: torch.Tensor, w16: torch.Tensor, K: int | None = None,
                 act: str | None = "silu", bias: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.float16, split_k: int = 0,
                 out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = act(x @ wg^T + bias_g) * (x @ wu^T + bias_u), in out_dtype (f16
    or f32), with w16 [2N, ld] the f16 caches of gate and up one after the
    other and bias f32 [2N] likewise; x as in linear_f16cache."""
    return _on_device(x, _binding().layer, "mq_glu_f16cache",
                      (x, w16, 0, -1, K, bias, _act(act), None, True,
                       _out_type(out_dtype), split_k, out, ws))


def glu_fused(x: torch.Tensor, wq: torch.Tensor, fmt, N: int, K: int | None = None,
              act: str | None = "silu", bias: torch.Tensor | None = None,
              out_dtype: torch.dtype = torch.float16, split_k: int = 0,
              out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """glu_f16cache straight from the quantized weights: wq holds the gate's N
    rows of K, then the up matrix's."""
    return _on_device(x, _binding().layer, "mq_glu_fused",
                      (x, wq, _fmt(fmt) or -1, N, K, bias, _act(act), None,
                       True, _out_type(out_dtype), split_k, out, ws))


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                 eps: float = 1e-6, out_dtype: torch.dtype = torch.float16,
                 out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None):
    """(y, h): h = x + residual, summed in f32 and rounded to the residual's type,
    and y [M, K] = h / sqrt(mean(h^2) + eps) * weight in out_dtype (f16 or f32;
    with out, in its type).

    x, residual [M, K] f32 or f16, any row stride from K on; weight f32 [K].
    Without a residual h is None and y the norm of x.  residual_out may be the residual
    itself (the stream is then updated in place)."""
    return _on_device(x, _binding().norm, "mq_add_rms_norm",
                      (x, weight, residual, eps, _out_type(out_dtype), out, None, residual_out))


def add_rms_norm_q8_1(x: torch.Tensor, weight: torch.Tensor,
                      residual: torch.Tensor | None = None, eps: float = 1e-6,
                      xq: torch.Tensor | None = None, ds: torch.Tensor | None = None,
                      residual_out: torch.Tensor | None = None):
    """(xq, ds, h): add_rms_norm with y as the int8 blocks that gemm_mmq reads,
    the ones quantize_q8_1 gives for the f32 y.  K a multiple of 32."""
    return _on_device(x, _binding().norm, "mq_add_rms_norm_q8_1",
                      (x, weight, residual, eps, -1, xq, ds, residual_out))
