"""Torch front end of the attention half of a layer: rotary positions, the 4-bit
key/value cache's store and load, and attention over it.

As in ``layers``: every step of the computation runs in the HIP library, one
native function (``csrc/binding_attention.cpp``) per operator checks, allocates
and calls, on the current stream of the tensors' device; all tensors of a call
are on one GPU, and results are not recorded by autograd (serving operators,
without a backward pass).

A batch is rows of one or more sequences over a paged cache.  ``table`` (int32 [B, W])
gives the page of each sequence's tokens, ``lens`` (int32 [B]) how many tokens each
has, the batch's own rows included: a sequence's n rows are its last n tokens.  They
are rows ``cu_rows[b]`` to ``cu_rows[b + 1]`` of the activations (int32 [B + 1]), or
without it equally many for each, in order.

Rows that are no sequence's (before ``cu_rows[0]``, behind ``cu_rows[B]``) are not written,
nor, by the store and the load, those of tokens before a sequence's first (``lens`` smaller
than its rows): a given output keeps there what it held, and a new one holds there what its
memory held.
"""

from __future__ import annotations

import ctypes
import math
import operator

import torch

from ._lib import MqKvQ4, check, lib
from .api import _as_int
from .layers import _binding, _on_device, _out_type

# pairs of a rotation (include/mq.h)
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def _layout(layout) -> int:
    code = ROPE_LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"unknown layout {layout!r}: one of {list(ROPE_LAYOUTS)}")
    return code


def rope_freqs(n_rot: int, base: float = 10000.0, scale: float = 1.0, factors=None,
               context: int | None = None, beta: tuple[float, float] = (1.0, 32.0),
               device=None) -> torch.Tensor:
    """The angle per position of each of n_rot/2 pairs, f64: base^(-2j/n_rot).

    For contexts ``scale`` times as long as those of training: divided by
    ``scale`` (position interpolation), and with ``context``, the length of
    training, only where a pair turns few times within it: r = context · f / 2π
    turns, weight w = clamp((r - beta[0]) / (beta[1] - beta[0]), 0, 1) of the plain
    frequency and 1 - w of the divided one.  (The magnitude that goes with that is
    0.1·ln(scale) + 1, ``mscale`` of the calls.)  ``factors``: n_rot/2 divisors of
    the frequencies, as some checkpoints carry them."""
    if n_rot <= 0 or n_rot % 2:
        raise ValueError(f"n_rot must be positive and even, got {n_rot}")
    if not (base > 0 and math.isfinite(base) and scale > 0 and math.isfinite(scale)):
        raise ValueError("base and scale must be positive and finite")
    f = base ** (-torch.arange(0, n_rot, 2, dtype=torch.float64) / n_rot)
    if factors is not None:
        d = torch.as_tensor(factors, dtype=torch.float64, device="cpu").reshape(-1)
        if d.numel() != n_rot // 2:
            raise ValueError(f"factors must be {n_rot // 2} values, got {d.numel()}")
        f = f / d
    if context is None:
        f = f / scale
    else:
        if not beta[1] > beta[0]:
            raise ValueError("beta must ascend")
        w = ((context * f / (2 * math.pi) - beta[0]) / (beta[1] - beta[0])).clamp(0, 1)
        f = w * f + (1 - w) * f / scale
    return f.to(device) if device is not None else f


def rope(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, head_dim: int,
         layout: str = "half", mscale: float = 1.0, out_dtype: torch.dtype | None = None,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """x [M, heads * head_dim] (f32 or f16, any row stride) with the first
    2 * len(freqs) elements of each head turned by the row's position (int32 [M]):
    pairs (j, j + len(freqs)), or (2j, 2j + 1) with layout "interleaved"; the rest
    copied.  freqs f64 on the GPU (rope_freqs).  In x's type, or out_dtype, or out's;
    out may be x itself."""
    return _on_device(x, _binding().rope, "mq_rope",
                      (x, positions, freqs, head_dim, _layout(layout), mscale,
                       -1 if out_dtype is None else _out_type(out_dtype), out))


def kv_page_bytes(heads: int, page: int, head_dim: int) -> int:
    """Bytes of one page of the 4-bit cache: heads * page * head_dim * 9 / 8."""
    return check(lib().mq_kv_q4_page_bytes(_as_int(heads), _as_int(page), _as_int(head_dim)),
                 "mq_kv_q4_page_bytes")


def kv_cache_q4(pages: int, heads: int, page: int, head_dim: int, device="cuda") -> torch.Tensor:
    """A cache for ``pages`` pages of ``page`` tokens (a multiple of 32) of ``heads``
    key/value heads of head_dim (64, 96, 128 or 256): uint8
    [pages, heads, page / 32, 36 * head_dim], zeros.  Pages may be strided (the
    layers of one allocation); the inner dimensions are contiguous."""
    kv_page_bytes(heads, page, head_dim)
    return torch.zeros((pages, heads, page // 32, 36 * head_dim), dtype=torch.uint8, device=device)


def kv_store_q4(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, table: torch.Tensor,
                lens: torch.Tensor, cu_rows: torch.Tensor | None = None,
                freqs: torch.Tensor | None = None, layout: str = "half", mscale: float = 1.0,
                positions: torch.Tensor | None = None, q: torch.Tensor | None = None,
                q_dtype: torch.dtype = torch.float16,
                q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Quantizes k and v [M, heads * head_dim] (f32 or f16) into the cache at the last
    positions of their sequences; with freqs the keys are rotated first (as rope
    does, by their positions in the sequence or by ``positions``, int32 [M]), and q
    [M, q_heads * head_dim] beside them.  A block of 32 with an element that is not finite
    or, rotated, beyond f16's range (65520 and more) reads back as NaN.  Returns the
    rotated q in q_dtype (or q_out, which may be q itself), None without q."""
    return _on_device(k, _binding().kv_store, "mq_kv_store_q4",
                      (k, v, cache, table, lens, cu_rows, freqs, _layout(layout), mscale, positions,
                       q, _out_type(q_dtype), q_out))


def kv_load_q4(cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, rows: int,
               cu_rows: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float16,
               k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None):
    """(k, v) [rows, heads * head_dim]: the keys and values of the batch's ``rows`` rows
    as the cache holds them, exact in f32, rounded once in f16."""
    return _on_device(cache, _binding().kv_load, "mq_kv_load_q4",
                      (cache, table, lens, rows, cu_rows, _out_type(out_dtype), k_out, v_out))


def attention_workspace_bytes(cache: torch.Tensor, batch: int, q_heads: int, rows: int,
                              max_len: int, ragged: bool = False) -> int:
    """Workspace bytes of attention_q4 for ``rows`` rows of ``batch`` sequences (ragged: with
    cu_rows), q_heads query heads and that max_len (the table's width times the
    page where the call gives none)."""
    if cache.dim() != 4 or cache.size(3) % 36:
        raise ValueError("cache must be [pages, heads, page / 32, 36 * head_dim]")
    max_len = operator.index(max_len)
    if not -(1 << 63) <= max_len < 1 << 63:   # (ctypes would pass its low 64 bits)
        raise OverflowError(f"max_len must fit in 64 bits, got {max_len}")
    one = 16   # an aligned address: the plan reads no memory
    kv = MqKvQ4(cache=one, page_bytes=1 << 62, pages=1, heads=_as_int(cache.size(1)),
                page=_as_int(32 * cache.size(2)), head_dim=_as_int(cache.size(3) // 36), table=one,
                table_width=1, table_ld=1, lens=one, cu_rows=one if ragged else None,
                batch=_as_int(batch))
    return check(lib().mq_attention_q4_workspace_bytes(ctypes.byref(kv), _as_int(q_heads),
                                                       _as_int(rows), max_len),
                 "mq_attention_q4_workspace_bytes")


def attention_q4(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                 cu_rows: torch.Tensor | None = None, scale: float | None = None,
                 causal: bool = True, window: int = 0, cap: float = 0.0,
                 slopes: torch.Tensor | None = None, prefix: torch.Tensor | None = None,
                 max_len: int | None = None, out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of q [M, q_heads * head_dim] (f32 or f16) over the cache, f16
    [M, q_heads * head_dim]; q_heads a multiple of the cache's heads.

    scale: of the scores (1/sqrt(head_dim)); cap > 0: scores become
    cap * tanh(score / cap); slopes (f32 [q_heads]): less slope * distance.  A row sees
    the tokens up to its own (all of its sequence's if not causal), with a window
    only those nearer than that, and always the first prefix[b] (int32 [B]).  Rows
    that see nothing are zeros.  max_len: a bound of lens where the table holds much
    more, for the launch plan.  ws: a workspace of attention_workspace_bytes.  The launch
    is planned for the mean number of rows: long prompts and single tokens are faster in
    a call each."""
    return _on_device(q, _binding().attend, "mq_attention_q4",
                      (q, cache, table, lens, cu_rows, scale, causal, window, cap, slopes, prefix,
                       max_len, out, ws))
