"""Torch front end of the operators around the quantized products: linear layers
(the product with bias, activation and residual in its epilogue), gated pairs of
them, and the residual RMS norm that feeds them.

As in ``api``, every step of the computation runs in the HIP library; these
functions check dtypes, devices, shapes and strides, allocate the outputs and
pass pointers on the current stream of the tensors' device.  All tensors of a
call must be on one GPU; it need not be the current one.
"""

from __future__ import annotations

import functools

import torch

from ._lib import MQ_F16, MQ_F32, check, lib
from .api import _fmt, _need_quant

_TYPES = {torch.float32: MQ_F32, torch.float16: MQ_F16}

# activations of a linear layer (include/mq.h)
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _type(t: torch.Tensor, name: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or float16, got {t.dtype}")
    return code


def _device(x: torch.Tensor, name: str) -> int:
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return dev


def _matrix(t: torch.Tensor, dev: int, rows: int, cols: int, name: str) -> int:
    """The row stride of a row-major matrix of at least rows x cols on GPU `dev`."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    if shape[0] < rows or shape[1] < cols:
        raise ValueError(f"{name} must be at least {rows} x {cols}, got {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same GPU as the activations")
    # the stride of a single row is never used
    return stride[0] if shape[0] > 1 else max(stride[0], cols)


def _vector(t: torch.Tensor, dev: int, n: int, name: str) -> int:
    """The address of a contiguous f32 vector of n elements on GPU `dev`."""
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be torch.float32, got {t.dtype}")
    if t.dim() != 1 or not t.is_contiguous() or t.shape[0] < n:
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same GPU as the activations")
    return t.data_ptr()


def _call(dev: int, name: str, *args) -> None:
    """lib().name(*args, stream) on GPU `dev`'s current stream, with `dev` current."""
    fn = getattr(lib(), name)
    if torch.cuda.current_device() == dev:
        check(fn(*args, torch.cuda.current_stream(dev).cuda_stream), name)
    else:
        with torch.cuda.device(dev):
            check(fn(*args, torch.cuda.current_stream(dev).cuda_stream), name)


def _act(act) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}: one of {list(ACTIVATIONS)}")
    return code


@functools.lru_cache(maxsize=4096)
def _layer_workspace(f: int, xt: int, M: int, N: int, K: int, split_k: int, glu: bool) -> int:
    name = "mq_glu_workspace_bytes" if glu else "mq_linear_workspace_bytes"
    return check(getattr(lib(), name)(f, xt, M, N, K, split_k), name)


def linear_workspace_bytes(fmt, M: int, N: int, K: int, split_k: int = 0, x_f32: bool = False,
                           glu: bool = False) -> int:
    """Workspace bytes of a linear layer (fmt 0 / "f16": the f16 cache), or with
    ``glu`` of a gated one with N output columns; x_f32 for f32 activations."""
    f = 0 if fmt in (0, None, "f16") else _fmt(fmt)
    return _layer_workspace(f, MQ_F32 if x_f32 else MQ_F16, int(M), int(N), int(K), int(split_k),
                            bool(glu))


def _layer(x, weight, f, N, K, act, bias, residual, glu, out_dtype, split_k, out, ws):
    """One linear (or gated) layer: f is 0 for an f16 cache, else the format of
    the quantized weight."""
    dev = _device(x, "x")
    xt = _type(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D with unit column stride")
    M = x.shape[0]
    rows = 2 * N if glu else N
    ldx = _matrix(x, dev, M, K, "x")
    if f:
        _need_quant(weight, f, rows, K)
        if weight.get_device() != dev:
            raise ValueError("wq must be on the same GPU as the activations")
        w = (f, weight.data_ptr())
    else:
        if weight.dtype != torch.float16:
            raise ValueError(f"w16 must be torch.float16, got {weight.dtype}")
        w = (weight.data_ptr(), _matrix(weight, dev, rows, K, "w16"))
    b = 0 if bias is None else _vector(bias, dev, rows, "bias")
    if glu:
        r = ()
    elif residual is None:
        r = (MQ_F32, 0, 0)
    else:
        ldr = _matrix(residual, dev, M, N, "residual")
        r = (_type(residual, "residual"), residual.data_ptr(), ldr)
    if out is None:
        if out_dtype not in _TYPES:
            raise ValueError(f"out_dtype must be float32 or float16, got {out_dtype}")
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
        ldy = N
    else:
        ldy = _matrix(out, dev, M, N, "out")
    yt = _type(out, "out")
    if ws is None:
        nbytes = _layer_workspace(f, xt, M, N, K, split_k, glu)
        if nbytes:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be contiguous, on the same GPU as the activations")
    wsp = (0, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    name = ("mq_glu_" if glu else "mq_linear_") + ("fused" if f else "f16cache")
    _call(dev, name, xt, x.data_ptr(), ldx, *w, b, _act(act), *r, yt, out.data_ptr(), ldy, M, N,
          K, *wsp, split_k)
    return out


def linear_f16cache(x: torch.Tensor, w16: torch.Tensor, K: int | None = None,
                    bias: torch.Tensor | None = None, act: str | None = None,
                    residual: torch.Tensor | None = None,
                    out_dtype: torch.dtype = torch.float32, split_k: int = 0,
                    out: torch.Tensor | None = None,
                    ws: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = act(x[:, :K] @ w16[:, :K]^T + bias) + residual, in out_dtype
    (f32 or f16): gemm_f16cache with the layer's epilogue.

    x [M, >=K] f16 (or f32, rounded to f16), w16 the f16 cache [N, ld], bias
    f32 [N], act one of ACTIVATIONS, residual [M, N] f32 or f16.  out may be
    the residual itself (the stream is then updated in place)."""
    K = x.shape[-1] if K is None else K
    return _layer(x, w16, 0, w16.shape[0], K, act, bias, residual, False, out_dtype, split_k, out,
                  ws)


def linear_fused(x: torch.Tensor, wq: torch.Tensor, fmt, N: int, K: int | None = None,
                 bias: torch.Tensor | None = None, act: str | None = None,
                 residual: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
                 split_k: int = 0, out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None) -> torch.Tensor:
    """linear_f16cache straight from the quantized weight wq [N rows of K]."""
    K = x.shape[-1] if K is None else K
    return _layer(x, wq, _fmt(fmt), N, K, act, bias, residual, False, out_dtype, split_k, out, ws)


def glu_f16cache(x: torch.Tensor, w16: torch.Tensor, K: int | None = None,
                 act: str | None = "silu", bias: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.float16, split_k: int = 0,
                 out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None) -> torch.Tensor:
    """y[M, N] = act(x @ wg^T + bias_g) * (x @ wu^T + bias_u), in out_dtype (f16
    or f32), with w16 [2N, ld] the f16 caches of gate and up one after the
    other and bias f32 [2N] likewise; x as in linear_f16cache."""
    if w16.shape[0] % 2:
        raise ValueError(f"w16 must have an even number of rows, got {w16.shape[0]}")
    K = x.shape[-1] if K is None else K
    return _layer(x, w16, 0, w16.shape[0] // 2, K, act, bias, None, True, out_dtype, split_k, out,
                  ws)


def glu_fused(x: torch.Tensor, wq: torch.Tensor, fmt, N: int, K: int | None = None,
              act: str | None = "silu", bias: torch.Tensor | None = None,
              out_dtype: torch.dtype = torch.float16, split_k: int = 0,
              out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """glu_f16cache straight from the quantized weights: wq holds the gate's N
    rows of K, then the up matrix's."""
    K = x.shape[-1] if K is None else K
    return _layer(x, wq, _fmt(fmt), N, K, act, bias, None, True, out_dtype, split_k, out, ws)


def _norm_inputs(x, weight, residual, residual_out):
    """(device, M, K, the library call's arguments up to H's stride but eps, h)."""
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D with unit column stride")
    M, K = x.shape
    ldx = _matrix(x, dev, M, K, "x")
    w = _vector(weight, dev, K, "weight")
    xt = _type(x, "x")
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return dev, M, K, (xt, x.data_ptr(), ldx, MQ_F32, 0, 0, w), (0, 0), None
    rt = _type(residual, "residual")
    ldr = _matrix(residual, dev, M, K, "residual")
    if residual_out is None:
        h = torch.empty((M, K), dtype=residual.dtype, device=x.device)
        ldh = K
    else:
        h = residual_out
        if h.dtype != residual.dtype:
            raise ValueError(f"residual_out must be {residual.dtype}, got {h.dtype}")
        ldh = _matrix(h, dev, M, K, "residual_out")
    return (dev, M, K, (xt, x.data_ptr(), ldx, rt, residual.data_ptr(), ldr, w),
            (h.data_ptr(), ldh), h)


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                 eps: float = 1e-6, out_dtype: torch.dtype = torch.float16,
                 out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None):
    """(y, h): h = x + residual in the residual's type, and y [M, K] = h /
    sqrt(mean(h^2) + eps) * weight in out_dtype (f16 or f32).

    x, residual [M, K] f32 or f16, any row stride; weight f32 [K].  Without a
    residual h is None and y the norm of x.  residual_out may be the residual
    itself (the stream is then updated in place)."""
    dev, M, K, head, tail, h = _norm_inputs(x, weight, residual, residual_out)
    if out is None:
        if out_dtype not in _TYPES:
            raise ValueError(f"out_dtype must be float32 or float16, got {out_dtype}")
        out = torch.empty((M, K), dtype=out_dtype, device=x.device)
        ldy = K
    else:
        ldy = _matrix(out, dev, M, K, "out")
    _call(dev, "mq_add_rms_norm", *head, eps, *tail, _type(out, "out"), out.data_ptr(), ldy, M, K)
    return out, h


def add_rms_norm_q8_1(x: torch.Tensor, weight: torch.Tensor,
                      residual: torch.Tensor | None = None, eps: float = 1e-6,
                      xq: torch.Tensor | None = None, ds: torch.Tensor | None = None,
                      residual_out: torch.Tensor | None = None):
    """(xq, ds, h): add_rms_norm with y as the int8 blocks that gemm_mmq reads,
    the ones quantize_q8_1 gives for the f32 y.  K a multiple of 32."""
    dev, M, K, head, tail, h = _norm_inputs(x, weight, residual, residual_out)
    if xq is None:
        xq = torch.empty((M, (K + 15) // 16 * 16), dtype=torch.int8, device=x.device)
    elif xq.dtype != torch.int8:
        raise ValueError(f"xq must be torch.int8, got {xq.dtype}")
    ldq = _matrix(xq, dev, M, K, "xq")
    if ds is None:
        ds = torch.empty((M, K // 32, 2), dtype=torch.float32, device=x.device)
    elif (ds.dtype != torch.float32 or not ds.is_contiguous() or ds.get_device() != dev
          or ds.numel() < M * (K // 32) * 2):
        raise ValueError("ds must be contiguous float32 with M*K/16 elements, on x's GPU")
    _call(dev, "mq_add_rms_norm_q8_1", *head, eps, *tail, xq.data_ptr(), ldq, ds.data_ptr(), M, K)
    return xq, ds, h
