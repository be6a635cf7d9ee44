"""Reference for the attention operators: rotary positions, the blocks and the
byte layout of the 4-bit key/value cache, and attention over it.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Rotation and attention are evaluated in binary64 from their definitions and
returned unrounded; the blocks follow the definition's f32 steps, bit for bit.
"""

from __future__ import annotations

import math

import numpy as np


def rotate_ref(x: np.ndarray, pos: np.ndarray, freqs: np.ndarray, layout: str = "half",
               mscale: float = 1.0) -> np.ndarray:
    """x [M, H, D] with the first 2·len(freqs) elements of every head turned."""
    y = np.asarray(x, dtype=np.float64).copy()
    n = len(freqs)
    a = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(freqs, dtype=np.float64)
    # cosine and sine of far angles: numpy's f64 argument reduction is exact
    c, s = np.cos(a)[:, None] * float(mscale), np.sin(a)[:, None] * float(mscale)
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else \
        (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    x0, x1 = y[..., first].copy(), y[..., second].copy()
    y[..., first] = x0 * c - x1 * s
    y[..., second] = x1 * c + x0 * s
    return y


def rotate_f32(x: np.ndarray, pos, freqs, layout: str = "half", mscale: float = 1.0) -> np.ndarray:
    """The rotation in its f32 steps: cosine and sine rounded to f32, then each
    product and sum."""
    y = np.asarray(x, dtype=np.float32).copy()
    n = len(freqs)
    a = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(freqs, dtype=np.float64)
    m = float(np.float32(mscale))
    c, s = ((f(a)[:, None] * m).astype(np.float32) for f in (np.cos, np.sin))
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else \
        (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    x0, x1 = y[..., first].copy(), y[..., second].copy()
    y[..., first] = x0 * c - x1 * s
    y[..., second] = x1 * c + x0 * s
    return y


def quantize_q4(x: np.ndarray):
    """(codes uint8, d as f16) of blocks of 32 along the last axis of f32 values."""
    b = np.asarray(x, dtype=np.float32)
    b = b.reshape(*b.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    mag = np.where(np.isfinite(b), np.abs(b), 0)
    at = mag.argmax(-1)                                   # the first of the largest
    top = np.take_along_axis(b, at[..., None], -1)[..., 0]
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        d = (top / np.float32(-8)).astype(np.float16)
        bad |= ~(np.abs(d.astype(np.float32)) <= 8188)   # d·(q − 8) has to be an f16 number
        df = d.astype(np.float32)[..., None]
        q = np.floor(b / df + np.float32(8.5))
    q = np.where((df == 0) | bad[..., None], 8, np.clip(np.nan_to_num(q), 0, 15))
    d = np.where(bad, np.float16(np.nan), np.where(d == 0, np.float16(0), d))
    return q.astype(np.uint8).reshape(*x.shape), d


def values(codes: np.ndarray, d: np.ndarray) -> np.ndarray:
    """What codes and scales stand for, in f64 (exact)."""
    with np.errstate(invalid="ignore"):
        return (codes.astype(np.float64) - 8) * np.repeat(d.astype(np.float64), 32, -1)


def cache_tokens(cache: np.ndarray, D: int):
    """The contents of a cache's bytes [pages, heads, tiles, 36·D], token by token:
    (key codes [pages, heads, page, D], key d [.., D/32], value codes, value d),
    one element at a time from the documented places."""
    P, H, T, _ = cache.shape
    NS = D // 32
    tiles = np.ascontiguousarray(cache)
    kc = tiles[..., :16 * D].copy().view("<u4")
    kd = tiles[..., 16 * D:18 * D].copy().view("<f2")
    vc = tiles[..., 18 * D:34 * D].copy().view("<u4")
    vd = tiles[..., 34 * D:].copy().view("<f2")
    out = (np.zeros((P, H, T * 32, D), np.uint8), np.zeros((P, H, T * 32, NS), np.float16),
           np.zeros((P, H, T * 32, D), np.uint8), np.zeros((P, H, T * 32, NS), np.float16))
    place = [4 * (e // 2) + 16 * (e % 2) for e in range(8)]
    for t in range(32):
        m, r = (t // 4) % 2, 4 * (t // 8) + t % 4
        for s in range(NS):
            out[1][:, :, t::32, s] = kd[..., (16 * m + r) * NS + s]
            out[3][:, :, t::32, s] = vd[..., (t // 8 * NS + s) * 8 + t % 8]
            for g in range(4):
                w = kc[..., ((4 * m + g) * 16 + r) * NS + s]
                for e in range(8):
                    out[0][:, :, t::32, 32 * s + 8 * g + e] = (w >> place[e]) & 15
        for d in range(D):
            out[2][:, :, t::32, d] = (vc[..., t // 8 * D + d] >> place[t % 8]) & 15
    return out


def visible_ref(positions, keys: int, causal: bool = True, window: int = 0,
                prefix: int = 0) -> np.ndarray:
    """[rows, keys]: which tokens the row at each position sees."""
    p, j = np.asarray(positions)[:, None], np.arange(keys)[None, :]
    see = (j <= p) if causal else np.ones((len(positions), keys), bool)
    if window:
        see = see & (np.abs(p - j) < window)
    return see | (j < prefix)


def attention_ref(q, k, v, positions, scale: float, causal=True, window=0, cap=0.0, slopes=None,
                  prefix=0):
    """(y, spread) of one sequence: q [n, H, D] at `positions`, k and v [len, Hkv, D], all
    in f64; spread = Σ softmax·|v|, what the roundings of the weights are proportional
    to.  A row that sees nothing is zeros; values of unseen tokens do not enter."""
    n, H, D = q.shape
    L, Hkv, _ = k.shape
    see = visible_ref(positions, L, causal, window, prefix)
    y = np.zeros((n, H, D))
    spread = np.zeros((n, H, D))
    dist = np.abs(np.asarray(positions, dtype=np.float64)[:, None] - np.arange(L)[None, :])
    with np.errstate(invalid="ignore", over="ignore"):
        for h in range(H):
            s = (q[:, h] @ k[:, h // (H // Hkv)].T) * scale
            if cap:
                s = cap * np.tanh(s / cap)
            if slopes is not None:
                s = s - float(slopes[h]) * dist
            for i in range(n):
                at = np.flatnonzero(see[i])
                if not len(at):
                    continue
                w = np.exp(s[i, at] - s[i, at].max())
                w /= w.sum()
                vs = v[at, h // (H // Hkv)]
                y[i, h] = w @ vs
                spread[i, h] = w @ np.abs(vs)
    return y, spread


def default_scale(D: int) -> float:
    return 1.0 / math.sqrt(D)
