"""Reference for the operators around the quantized products: the residual RMS
norm, and a linear layer's epilogue (bias, activation, residual) with its gated
pair.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Everything is evaluated in binary64 from the definition; results are returned
in binary64, unrounded, so that a test states each rounding of the operator as
a tolerance of its own.
"""

from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def rms_norm_ref(x: np.ndarray, w: np.ndarray, eps: float, r: np.ndarray | None = None):
    """(y, h) in f64: h = x + r, rounded once to r's dtype as the stored stream
    is (h = x without r), y = h / sqrt(mean(h²) + eps) · w."""
    h = np.asarray(x, dtype=np.float64)
    if r is not None:
        # the f32 sum is rounded to the stream's type in a second step when
        # that is f16
        h = (h + np.asarray(r, dtype=np.float64)).astype(np.float32).astype(r.dtype)
        h = h.astype(np.float64)
    inv = 1.0 / np.sqrt((h * h).mean(axis=-1, keepdims=True) + float(eps))
    return h * inv * np.asarray(w, dtype=np.float64), h


def act_ref(v: np.ndarray, act: str) -> np.ndarray:
    """The activation in f64."""
    v = np.asarray(v, dtype=np.float64)
    if act == "none":
        return v
    if act == "relu":
        return np.where(v < 0, 0.0, v)
    if act == "silu":
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-v))
    if act == "gelu":
        erfc = np.vectorize(math.erfc, otypes=[np.float64])
        return 0.5 * v * erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-2.0 * u))     # 0.5·v·(1 + tanh u)
    raise ValueError(act)


def linear_ref(x_bits, w_bits, K: int, bias=None, act: str = "none", residual=None):
    """(y, S): act(X·Wᵀ + bias) + residual in f64, and S = |X|·|W|ᵀ + |bias|, what
    the f32 sums of the product are proportional to."""
    from .gemm import gemm_ref

    v, S = gemm_ref(x_bits, w_bits, K)
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        v, S = v + b, S + np.abs(b)
    y = act_ref(v, act)
    if residual is not None:
        y = y + np.asarray(residual, dtype=np.float64)
    return y, S


def glu_ref(x_bits, w_bits, K: int, bias=None, act: str = "silu"):
    """(y, g, u, Sg, Su): act(g) · u with [g | u] = X·Wᵀ + bias, the first half of
    W's rows being the gate's."""
    from .gemm import gemm_ref

    v, S = gemm_ref(x_bits, w_bits, K)
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        v, S = v + b, S + np.abs(b)
    n = v.shape[1] // 2
    g, u = v[:, :n], v[:, n:]
    return act_ref(g, act) * u, g, u, S[:, :n], S[:, n:]
