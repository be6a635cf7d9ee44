"""The reference of the attention operators pinned by hand-derived cases (CPU)."""

import math

import numpy as np
import pytest

from oracle import attention as oa


def test_rotation_by_quarter_turns():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    f = np.array([math.pi / 2, math.pi])
    y = oa.rotate_ref(x, [1], f, "half")                 # pairs (0, 2), (1, 3)
    assert np.allclose(y, [[[-3, -2, 1, -4, 5]]], atol=1e-15)
    y = oa.rotate_ref(x, [1], f, "interleaved", 2.0)     # pairs (0, 1), (2, 3)
    assert np.allclose(y, [[[-4, 2, -6, -8, 5]]], atol=1e-15)
    back = oa.rotate_ref(oa.rotate_ref(x, [7], f / 3), [-7], f / 3)
    assert np.allclose(back, x, atol=1e-14)


def test_rotation_keeps_relative_positions():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f = 10000.0 ** (-np.arange(32) / 32)
    dots = [float((oa.rotate_ref(q, [p + 5], f) * oa.rotate_ref(k, [p], f)).sum())
            for p in (0, 100, 1000000)]
    assert np.allclose(dots, dots[0], atol=1e-8)


def test_f32_rotation_is_near():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 16)).astype(np.float32)
    f = 10000.0 ** (-np.arange(8) / 8)
    for layout in ("half", "interleaved"):
        a = oa.rotate_ref(x, [0, 9, 500000], f, layout)
        b = oa.rotate_f32(x, [0, 9, 500000], f, layout)
        assert b.dtype == np.float32 and np.abs(a - b).max() < 8 * 2.0 ** -24


def test_blocks_by_hand():
    b = np.zeros(32, np.float32)
    b[3], b[5], b[6], b[7], b[8] = -8, 7, 0.5, 0.49, 8
    q, d = oa.quantize_q4(b)
    assert d[0] == 1 and q[3] == 0 and q[5] == 15 and q[6] == 9 and q[7] == 8 and q[8] == 15
    assert q[0] == 8
    q, d = oa.quantize_q4(-b)                            # the first of the largest decides
    assert d[0] == -1 and q[3] == 0 and q[5] == 15 and q[6] == 9
    z, d = oa.quantize_q4(np.zeros(64, np.float32))
    assert (z == 8).all() and (d == 0).all()
    for bad in (np.nan, np.inf, -np.inf, 1e6):           # 1e6 / 8 overflows f16
        c = b.copy()
        c[9] = bad
        q, d = oa.quantize_q4(c)
        assert np.isnan(d[0]) and (q == 8).all()


def test_blocks_end_where_f16_does():
    """65504 = 8 · 8188 is f16's largest number; 65520 is the first that rounds beyond it."""
    b = np.linspace(-1000, 1000, 32, dtype=np.float32)
    for sign in (-1, 1):
        for top in (65504.0, 65519.0, np.nextafter(np.float32(65520), np.float32(0))):
            b[9] = sign * top
            q, d = oa.quantize_q4(b)
            assert d[0] == -sign * 8188 and q[9] == 0
            assert np.isfinite(oa.values(q, d).astype(np.float16)).all()
        for top in (65520.0, 65536.0, 1e5, 524000.0):     # of these d alone would be finite
            b[9] = sign * top
            q, d = oa.quantize_q4(b)
            assert np.isnan(d[0]) and (q == 8).all()


def test_blocks_are_within_half_a_step():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((50, 96)).astype(np.float32)
    q, d = oa.quantize_q4(x)
    step = np.abs(np.repeat(d.astype(np.float64), 32, -1))
    err = np.abs(oa.values(q, d) - x)
    # half a step, and at the far end, where 8 steps would be code 16, a whole one;
    # d's own rounding moves the 8 steps by 8·2^-11
    assert (err <= step * (1 + 2.0 ** -7)).all()
    assert (err <= step * (0.5 + 2.0 ** -7))[q < 15].all()


@pytest.mark.parametrize("D", [64, 96])
def test_cache_layout_round_trip(D):
    """Codes put at the documented places come back from them."""
    rng = np.random.default_rng(D)
    raw = rng.integers(0, 256, (2, 3, 2, 36 * D), dtype=np.uint8)
    kc, kd, vc, vd = oa.cache_tokens(raw, D)
    # every nibble and every scale once
    assert kc.shape == (2, 3, 64, D) and vd.shape == (2, 3, 64, D // 32)
    for codes, lo in ((kc, 0), (vc, 18 * D)):
        part = raw[..., lo:lo + 16 * D]
        want = np.bincount(np.concatenate((part.ravel() & 15, part.ravel() >> 4)), minlength=16)
        assert np.array_equal(np.bincount(codes.ravel(), minlength=16), want)
    for d, lo in ((kd, 16 * D), (vd, 34 * D)):
        part = np.ascontiguousarray(raw[..., lo:lo + 2 * D]).view("<u2")
        assert np.array_equal(np.sort(d.view(np.uint16).ravel()), np.sort(part.ravel()))
    # three places by hand: key token 13 = 8·1 + 4·1 + 1 is m = 1, r = 5
    w = np.ascontiguousarray(raw[0, 1, 0]).view("<u4")
    assert kc[0, 1, 13, 8 * 2 + 5] == (w[((4 * 1 + 2) * 16 + 5) * (D // 32)] >> 24) & 15
    assert vc[0, 1, 13, 7] == (w[18 * D // 4 + D + 7] >> 24) & 15        # octet 1, token 5 of it
    assert vc[1, 2, 63, D - 1] == \
        (np.ascontiguousarray(raw[1, 2, 1]).view("<u4")[18 * D // 4 + 4 * D - 1] >> 28) & 15


def test_visible():
    see = oa.visible_ref([-1, 0, 3], 6, True, 0, 0).astype(int).tolist()
    assert see == [[0] * 6, [1, 0, 0, 0, 0, 0], [1, 1, 1, 1, 0, 0]]
    assert oa.visible_ref([4], 6, True, 2, 1)[0].astype(int).tolist() == [1, 0, 0, 1, 1, 0]
    assert oa.visible_ref([2], 6, False, 2, 0)[0].astype(int).tolist() == [0, 1, 1, 1, 0, 0]


def test_attention_by_hand():
    # one head of one element: scores 0 and ln 3, weights 1/4 and 3/4
    q, k, v = np.array([[[1.0]]]), np.array([[[0.0]], [[math.log(3)]]]), np.array([[[4.0]], [[-8.0]]])
    y, s = oa.attention_ref(q, k, v, [1], 1.0)
    assert np.allclose(y, -5) and np.allclose(s, 7)
    y, _ = oa.attention_ref(q, k, v, [0], 1.0)
    assert np.allclose(y, 4)
    y, _ = oa.attention_ref(q, k, v, [-1], 1.0)
    assert (y == 0).all()
    y, _ = oa.attention_ref(q, k, v, [1], 1.0, slopes=[math.log(3)])     # token 0 is 1 away
    assert np.allclose(y, (4 - 8 * 9) / 10)
    c = 0.5
    w = math.exp(c * math.tanh(math.log(3) / c))
    y, _ = oa.attention_ref(q, k, v, [1], 1.0, cap=c)
    assert np.allclose(y, (4 - 8 * w) / (1 + w))
    v[0] = np.nan                                        # an unseen NaN stays out
    y, _ = oa.attention_ref(q, k, v, [1], 1.0, window=1)
    assert np.allclose(y, -8)
