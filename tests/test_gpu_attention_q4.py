"""Attention over the 4-bit cache on the GPU against the f64 oracle, on the values that
the cache holds (exact, through the load).

Tolerance, per output element; e = 2^-11 is f16's half step, u = 2^-24.
  scores   k enters exactly, as two f16 numbers (7 and 4 bits of the scale times the code);
           f32 queries as two as well, of which the product of the low parts is left out
           (2^-11 · 2^-7 of the product) and what is below 2^-24 (half a step, 2^-25·Σ|k|).
           At most 3·D products are summed in f32 ((3D)·u of Σ|q·k|), and scaling, cap, bias
           and the exponent's argument round a few times more; a cap of at most 128 adds
           2^-21 of it (1/(1 + e^2u) is good to 2^-22 and counts twice the cap).
           δ = scale·max_j Σ|q·k_j|·(2^-18 [f32] + (3D + 16)·u) + scale·2^-25·max_j Σ|k_j| [f32]
             + 8u·(max_j|s_j| + cap), and the hardware's exponential adds 2u: a weight and the
           sum of weights are each off by at most e^(δ + 2u) − 1
  output   values enter as f16: e of Σ w|v|; weights as two f16 numbers: 2^-22 of it; the
           sums of L terms in f32, L·u; weights are held to 2^-32 of the largest (f16 at 2^7
           and more for it): L·2^-32·max|v|
  rounding e of the value, 2^-25 below the smallest normal
Together: S·(2·(e^(δ + 2u) − 1)·1.01 + (e + 2^-21)·1.01 + 2·L·u) + L·2^-32·max|v| + e·|y| + 2^-25, S =
Σ w|v|."""

import numpy as np
import pytest

from gpu_common import announce, dev, needs_gpu, to_host
from oracle import attention as oa

pytestmark = [pytest.mark.gpu, needs_gpu]

import torch  # noqa: E402

import quantized_weight_prefill_q4_amd as mq  # noqa: E402
from test_gpu_kv_q4 import Batch, ints, rows_of  # noqa: E402

T = {"f32": torch.float32, "f16": torch.float16}
E, U = 2.0 ** -11, 2.0 ** -24


def filled(D, Hkv, page, rows, lens, seed=0, ragged=True, stride=0, gain=1.0):
    """A batch whose sequences' tokens are all in the cache (behind them: NaN scales)."""
    s = Batch(D, Hkv, page, rows, lens, seed, ragged, stride)
    k, v = (rows_of(sum(lens), Hkv * D, torch.float16, 100 + seed + i) for i in (0, 1))
    cu = ints(np.concatenate(([0], np.cumsum(lens))).tolist())
    mq.kv_store_q4(k * gain, v, s.cache, s.table, s.lens_t, cu_rows=cu)
    s.k, s.v = (to_host(t).astype(np.float64).reshape(-1, Hkv, D) for t in
                mq.kv_load_q4(s.cache, s.table, s.lens_t, sum(lens), cu_rows=cu,
                              out_dtype=torch.float32))
    s.tok = np.concatenate(([0], np.cumsum(lens)))
    return s


def expect(s, q, H, b, positions, rows, scale, causal, window, cap, slopes, prefix, keys=None,
           wide=False):
    """(y, tolerance) of sequence b's rows."""
    D = s.D
    at = slice(s.tok[b], s.tok[b + 1]) if keys is None else np.asarray(keys) + s.tok[b]
    k, v = s.k[at], s.v[at]
    qq = q[rows]
    y, S = oa.attention_ref(qq, k, v, positions, scale, causal, window, cap, slopes, prefix)
    tol = np.zeros_like(y)
    L = len(k)
    if L:
        G = H // s.Hkv
        dist = np.abs(np.asarray(positions, dtype=np.float64)[:, None] - np.arange(L)[None, :]).max()
        for h in range(H):
            big = abs(scale) * (np.abs(qq[:, h]) @ np.abs(np.nan_to_num(k[:, h // G])).T).max(1)
            top = big + (abs(slopes[h]) * dist if slopes is not None else 0)
            delta = big * ((3 * D + 16) * U + (2.0 ** -18 if wide else 0)) + 8 * U * (top + cap) + 2 * U
            if wide:
                delta = delta + abs(scale) * 2.0 ** -25 * np.abs(np.nan_to_num(k[:, h // G])).sum(1).max()
            w = 2 * np.expm1(np.minimum(delta, 50)) * 1.01 + (E + 2.0 ** -21) * 1.01 + 2 * L * U
            tol[:, h] = S[:, h] * w[:, None] + L * 2.0 ** -32 * np.abs(np.nan_to_num(v)).max()
    return y, tol + E * np.abs(y) + 2.0 ** -25


def check(s, H, xt="f16", seed=1, pad=0, lead=0, gain=1.0, causal=True, window=0, cap=0.0,
          slopes=None, prefix=None, scale=None, max_len=None):
    announce("attention_q4", "D", s.D, "H", H, s.Hkv, "page", s.page, "rows", s.rows[:8], "lens",
             s.lens[:8], xt, dict(pad=pad, causal=causal, window=window, cap=cap,
                                  slopes=slopes is not None, prefix=prefix, max_len=max_len))
    W = H * s.D
    q = rows_of(s.M, W, T[xt], seed, pad, lead) * gain
    if pad:
        buf = torch.full((s.M, W + pad), float("nan"), dtype=q.dtype, device=dev())
        buf[:, :W] = q
        q = buf[:, :W]
    sl = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device=dev())
    pf = None if prefix is None else ints(prefix)
    out = torch.full((s.M, W + pad), 77.0, dtype=torch.float16, device=dev())
    y = mq.attention_q4(q, s.cache, s.table, s.lens_t, cu_rows=s.cu, scale=scale, causal=causal,
                        window=window, cap=cap, slopes=sl, prefix=pf, max_len=max_len,
                        out=out[:, :W])
    assert bool((out[:, W:] == 77).all())
    qs = to_host(q).astype(np.float64).reshape(s.M, H, s.D)
    got = to_host(y).astype(np.float64).reshape(s.M, H, s.D)
    sc = oa.default_scale(s.D) if scale is None else scale
    worst = 0.0
    for b, (r, n) in enumerate(zip(s.rows, s.lens)):
        if not r:
            continue
        rows = slice(s.cu_np[b], s.cu_np[b] + r)
        ref, tol = expect(s, qs, H, b, np.arange(n - r, n), rows, sc, causal, window, cap, slopes,
                          0 if prefix is None else min(max(prefix[b], 0), n),
                          wide=xt == "f32")
        ratio = np.abs(got[rows] - ref) / tol
        assert np.isfinite(got[rows]).all(), b
        worst = max(worst, float(ratio.max()))
    assert worst <= 1, f"{worst:.3g} times its tolerance"
    return q, y


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_single_tokens(D, group):
    lens = [1, 2, 31, 32, 33, 63, 64, 65, 127, 200, 1000]
    s = filled(D, 2, 32, [1] * len(lens), lens, seed=D, ragged=False)
    check(s, 2 * group)
    check(s, 2 * group, xt="f32", gain=3.0)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("rows", [[2, 5, 1], [16, 17, 3], [33, 1, 70], [130, 0, 64]])
def test_several_rows(D, rows):
    lens = [r + p for r, p in zip(rows, (0, 45, 300))]
    s = filled(D, 2, 64, rows, lens, seed=sum(rows))
    check(s, 4)
    check(s, 14, xt="f32", causal=False)


def test_one_sequence_of_many_rows_among_single_tokens():
    """The kernel for few rows on a sequence of many: its row tiles share their parts."""
    s = filled(128, 2, 32, [150] + [1] * 30, [700] + [40 + b for b in range(30)], seed=41)
    check(s, 8)
    check(s, 8, xt="f32", window=60)
    s = filled(64, 1, 64, [1, 90, 2, 1, 0, 1], [3, 3000, 200, 1, 7, 64], seed=42)
    check(s, 1, prefix=[130] * 6)


@pytest.mark.parametrize("length", [2000, 5003, 20000])
def test_long_sequences_in_parts(length):
    s = filled(128, 2, 256, [1], [length], seed=length % 97, ragged=False)
    q, y = check(s, 14, gain=2.0)
    for limit in (0, 40, 1000, 1 << 40):        # the plan's bound changes the parts alone
        check(s, 14, gain=2.0, max_len=limit)
    s = filled(64, 1, 32, [3, 1], [length, 17], seed=length % 89)
    check(s, 8, xt="f32")


def test_many_and_unequal_sequences():
    """More sequences than lanes of a wave, empty ones among them, and one much longer than
    the others: the keys are dealt out over the batch."""
    rng = np.random.default_rng(3)
    rows = [int(r) for r in rng.integers(0, 4, 150)]
    lens = [r + int(p) for r, p in zip(rows, rng.integers(0, 400, 150))]
    s = filled(64, 1, 32, rows, lens, seed=21)
    check(s, 5)
    check(s, 5, xt="f32", window=100, max_len=100)
    lens = [int(n) for n in rng.integers(1, 90, 70)]
    s = filled(64, 2, 32, [1] * 70, lens, seed=22, ragged=False)
    check(s, 4, max_len=1 << 20)
    for at in (0, 30, 66):
        lens[at] = 9000
        s = filled(64, 1, 64, [1] * 67, lens[:67], seed=23 + at, ragged=False)
        check(s, 4)
        lens[at] = 50


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("rows", [11, 16, 22, 32, 33, 43])
def test_between_few_and_many_rows(D, rows):
    s = filled(D, 2, 32, [rows] * 2, [rows + 37, 1800], seed=rows + D, ragged=False)
    check(s, 6)                                    # 33 to 99 rows of a key/value head
    check(s, 6, max_len=1000)
    check(s, 6, xt="f32", window=500, slopes=[0.1] * 6)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_many_rows_in_parts(D):
    s = filled(D, 1, 64, [70], [1700], seed=31 + D, ragged=False)
    check(s, 4)
    check(s, 4, xt="f32", causal=False, max_len=100)
    check(s, 4, causal=False)
    s = filled(D, 2, 32, [100, 3, 40], [2100, 3, 900], seed=32 + D)
    check(s, 6)
    check(s, 6, xt="f32", cap=20.0, window=700)
    s = filled(D, 1, 32, [8], [6000], seed=33 + D, ragged=False)     # few jobs, many parts
    check(s, 16)


@pytest.mark.parametrize("D,rows,lens", [(128, [1, 1, 1], [300, 40, 1]), (96, [40, 7], [333, 7]),
                                         (256, [20, 3], [150, 90]), (64, [200], [200])])
@pytest.mark.parametrize("kw", [
    dict(window=1), dict(window=33), dict(window=128, causal=False), dict(window=2, causal=False),
    dict(cap=5.0), dict(cap=1000.0, gain=4.0), dict(cap=1e-39), dict(cap=1.0, scale=1e36), dict(slopes=True), dict(slopes=True, causal=False),
    dict(prefix=20), dict(prefix=20, window=16), dict(prefix=10000), dict(prefix=-4),
    dict(causal=False), dict(scale=0.0), dict(scale=-0.3),
    dict(window=40, cap=3.0, slopes=True, prefix=37)])
def test_masks_and_scores(D, rows, lens, kw):
    s = filled(D, 2, 32, rows, lens, seed=D + len(rows))
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = [2.0 ** (-(h + 1)) for h in range(6)]
    if "prefix" in kw:
        kw["prefix"] = [kw["prefix"]] * len(rows)
    check(s, 6, **kw)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("rows", [3, 100])             # few and many rows of a key/value head
@pytest.mark.parametrize("kw", [
    dict(scale=1.0), dict(scale=-1.0), dict(scale=0.7), dict(scale=1.0, slopes=True),
    dict(cap=1.0, scale=1e36), dict(cap=3.0, scale=-1e30), dict(cap=1e-39, scale=0.5),
    dict(cap=1e-3, scale=1e-4), dict(cap=8.0, scale=0.02), dict(cap=128.0, scale=0.5),
    dict(cap=129.0, scale=0.5), dict(cap=1000.0, scale=0.5), dict(cap=5000.0, scale=1e-3),
    dict(cap=50.0, scale=0.05, slopes=True, window=40)])
def test_scores_that_f32_sums_exactly(D, rows, kw):
    """Queries and keys of small whole numbers: every sum of products is exact, so that the
    tolerance holds what scale, cap, bias and exponential round and nothing else:
      δ = 8u·(max|s| + cap) + 2^-21·cap [tanh's quotient: 2/(1 + e) within 2^-21.8 of 1] + 2u,
    at most 2^-9, far from letting a wrong sign, cap or maximum pass."""
    announce("attention_q4 exact sums", D, rows, kw)
    H, Hkv, n = 4, 2, rows + 61
    rng = np.random.default_rng(D + rows)
    s = Batch(D, Hkv, 32, [rows], [n], D, False)
    k = rng.integers(-7, 8, (n, Hkv * D)).astype(np.float32)
    k[:, ::32] = -8                                    # so d is 1 and the codes are the numbers
    v = rows_of(n, Hkv * D, torch.float32, 9)
    mq.kv_store_q4(torch.from_numpy(k).to(dev()), v, s.cache, s.table, s.lens_t)
    lk, lv = mq.kv_load_q4(s.cache, s.table, s.lens_t, n, out_dtype=torch.float32)
    s.k, s.v = (to_host(t).astype(np.float64).reshape(n, Hkv, D) for t in (lk, lv))
    assert np.array_equal(s.k.reshape(n, -1), k)
    q = rng.integers(-3, 4, (rows, H * D))
    qs = q.astype(np.float64).reshape(rows, H, D)
    a = dict(cap=0.0, slopes=None, window=0) | kw
    if a["slopes"]:
        a["slopes"] = [0.5, 0.25, 2.0, 0.125]
    a["scale"] = float(np.float32(a["scale"]))
    a["cap"] = float(np.float32(a["cap"]))
    at = np.arange(n - rows, n)
    y, S = oa.attention_ref(qs, s.k, s.v, at, a["scale"], True, a["window"], a["cap"], a["slopes"], 0)
    top = max(float(np.abs(qs[:, h] @ s.k[:, h // 2].T).max()) for h in range(H)) * abs(a["scale"])
    if a["cap"]:
        top = min(top, a["cap"])
    top += 2.0 * n if a["slopes"] else 0
    delta = 8 * U * (top + a["cap"]) + 2.0 ** -21 * a["cap"] + 2 * U
    assert delta <= (2.0 ** -9 if a["cap"] <= 1000 else 2.0 ** -7)
    tol = S * (2 * np.expm1(delta) * 1.01 + (E + 2.0 ** -21) * 1.01 + 2 * n * U) + \
        n * 2.0 ** -32 * np.abs(s.v).max() + E * np.abs(y) + 2.0 ** -25
    sl = None if a["slopes"] is None else torch.tensor(a["slopes"], device=dev())
    for xt in ("f16", "f32"):
        got = mq.attention_q4(torch.from_numpy(q).to(dev()).to(T[xt]), s.cache, s.table, s.lens_t,
                              scale=a["scale"], cap=a["cap"], window=a["window"], slopes=sl)
        err = np.abs(to_host(got).astype(np.float64).reshape(rows, H, D) - y)
        assert (err <= tol).all(), (xt, float((err / tol).max()))


def test_large_and_small_scores():
    """Scores far apart and far from 0: the running maximum and its rescaling."""
    s = filled(128, 1, 32, [1, 9], [700, 150], seed=5, gain=20.0)
    check(s, 4, gain=8.0)
    check(s, 4, gain=1e-3)
    check(s, 4, gain=8.0, scale=1.0)
    s = filled(128, 1, 32, [1, 70], [300, 150], seed=6, gain=1e-5)     # scales below f16's normals
    for xt in ("f16", "f32"):
        check(s, 4, xt=xt, scale=2e4)
    check(s, 4, xt="f32", gain=1e-4, scale=1e8)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("rows", [1, 5, 40, 200])
def test_f32_queries_of_any_magnitude(D, rows):
    """Queries times a power of two, with the scale divided by it, give the same bits: f16's
    range does not show, whatever the other rows of the call are like (of other rows' scores
    the moments follow at which sums are rescaled: results are then within the tolerance)."""
    announce("attention_q4 f32 queries of any magnitude", D, rows)
    s = filled(D, 2, 32, [rows], [rows + 50], seed=3, ragged=False)
    kw = [dict(), dict(cap=5.0), dict(cap=500.0, slopes=torch.ones(4, device=dev()))]
    q, y = check(s, 4, xt="f32", scale=0.125, seed=5)
    run = lambda q, scale, kw: mq.attention_q4(q, s.cache, s.table, s.lens_t, scale=scale, **kw)
    want = [run(q, 0.125, k) for k in kw]
    assert torch.equal(want[0], y)
    qs = to_host(q).astype(np.float64).reshape(rows, 4, D)
    ref, tol = expect(s, qs, 4, 0, np.arange(50, rows + 50), slice(0, rows), 0.125, True, 0, 0.0,
                      None, 0, wide=True)

    def near(t, mine):
        got = to_host(t).astype(np.float64).reshape(rows, 4, D)
        return bool((np.abs(got - ref) <= tol)[mine].all())

    powers = (-110, -60, -30, -15, -4, 3, 12, 20, 60, 110)
    for p in powers:
        for k, w in zip(kw, want):
            assert torch.equal(run(q * 2.0 ** p, 2.0 ** (-3 - p), k), w), (p, k)
    if rows > 1:
        own = [powers[i % len(powers)] for i in range(rows)]
        mixed = q * torch.tensor([2.0 ** p for p in own], device=dev())[:, None]
        for p in powers:
            mine = [i for i in range(rows) if own[i] == p]
            # (rows of a larger magnitude: scores far beyond 2^24, nobody's result)
            assert near(run(mixed, 2.0 ** (-3 - p), {}), mine), p
    # the elements of a row far below its largest: what they contribute is below its last bits
    tiny = q.clone()
    tiny[:, 1::2] *= 2.0 ** -60
    none = q.clone()
    none[:, 1::2] = 0
    assert torch.equal(run(tiny, 0.125, {}), run(none, 0.125, {}))
    # rows of zeros, and of one infinity or NaN
    odd = q.clone()
    odd[0] = 0
    if rows > 2:
        odd[1, 3], odd[2, D + 3] = float("inf"), float("nan")
    z = run(odd, 0.125, {})
    assert bool(torch.isfinite(z[0]).all())
    if rows > 2:
        assert near(z, slice(3, rows))
        bad = ~torch.isfinite(z.view(rows, 4, D))
        assert bool(bad[1, 0].all()) and bool(bad[2, 1].all())
        bad[1, 0] = bad[2, 1] = False
        assert not bool(bad.any())


def test_other_streams_and_two_graphs_on_one_workspace():
    """Two captured calls of different kernels share a workspace; each replay is compared."""
    announce("attention_q4 two graphs, one workspace")
    D, H = 128, 8
    s1 = filled(D, 2, 64, [1, 1, 1], [3000, 5, 1200], seed=51)
    s2 = filled(D, 2, 64, [90, 20], [2000, 700], seed=52)
    q1, q2 = (rows_of(s.M, H * D, torch.float16, 53) for s in (s1, s2))
    need = [mq.attention_workspace_bytes(s.cache, len(s.lens), H, s.M, 4096, ragged=True)
            for s in (s1, s2)]
    assert min(need) > 0
    ws = torch.full((max(need),), 255, dtype=torch.uint8, device=dev())
    run = [lambda s=s, q=q: mq.attention_q4(q, s.cache, s.table, s.lens_t, cu_rows=s.cu,
                                            max_len=4096, ws=ws) for s, q in ((s1, q1), (s2, q2))]
    eager = [f().clone() for f in run]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for f, y in zip(run, eager):
            assert torch.equal(f(), y)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f in run:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = f()
        graphs.append((g, y))
    for _ in range(4):
        for (g, y), want in zip(graphs, eager):
            y.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
            run[1]()
            ws.fill_(255)
    # shorter sequences between replays: the parts follow the lengths on the device
    s1.lens_t.copy_(ints([40, 5, 900]))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    got = graphs[0][1].clone()
    assert torch.equal(got, run[0]())


def test_strides_and_odd_rows():
    for xt in ("f16", "f32"):
        s = filled(64, 3, 96, [5, 30], [5, 130], seed=6, stride=48)
        check(s, 9, xt=xt, pad=1)
        check(s, 3, xt=xt, pad=512)


def test_lists_beside_the_outputs():
    """Outputs may not overlap the lists that a call reads, but one buffer may hold both: lists
    in the columns between an output's rows, and right behind its last."""
    announce("lists beside the outputs")
    D, H, M = 64, 4, 3
    s = filled(D, 2, 32, [1] * M, [40, 3, 65], seed=44, ragged=False)
    q = rows_of(M, H * D, torch.float16, 45)
    f = mq.rope_freqs(D, device=dev())
    k, v = rows_of(M, 2 * D, torch.float16, 46), rows_of(M, 2 * D, torch.float16, 47)
    row = H * D + 16
    y = mq.attention_q4(q, s.cache, s.table, s.lens_t)
    buf = torch.zeros(M * row + 4 * s.table.numel(), dtype=torch.float16, device=dev())
    out = buf[:M * row].view(M, row)[:, :H * D]
    lens = buf[H * D:H * D + 2 * M].view(torch.int32)       # between rows 0 and 1
    table = buf[M * row - 16:M * row - 16 + 2 * s.table.numel()].view(torch.int32).view_as(s.table)
    lens.copy_(s.lens_t)
    table.copy_(s.table)
    assert torch.equal(mq.attention_q4(q, s.cache, table, lens, out=out), y)
    want = mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t, freqs=f, q=q)
    bytes1 = s.bytes.clone()
    assert torch.equal(mq.kv_store_q4(k, v, s.cache, table, lens, freqs=f, q=q, q_out=out), want)
    assert torch.equal(s.bytes, bytes1)
    lk, lv = mq.kv_load_q4(s.cache, s.table, s.lens_t, M)
    mq.kv_load_q4(s.cache, table, lens, M, k_out=out[:, :2 * D], v_out=out[:, 2 * D:])
    assert torch.equal(out, torch.cat((lk, lv), 1))
    assert torch.equal(lens, s.lens_t) and torch.equal(table, s.table)
    # lists between the pages of a strided cache
    p = Batch(D, 2, 32, [1] * M, [40, 3, 65], 44, False, stride=4096)
    p.bytes[:, :-4096] = s.bytes
    gap = p.bytes[0, -4096:].view(torch.int32)
    lens2, table2 = gap[:M], gap[64:64 + s.table.numel()].view_as(s.table)
    lens2.copy_(s.lens_t)
    table2.copy_(s.table)
    assert torch.equal(mq.kv_store_q4(k, v, p.cache, table2, lens2, freqs=f, q=q), want)
    assert torch.equal(p.bytes[:, :-4096], s.bytes) and torch.equal(table2, s.table)
    assert torch.equal(mq.attention_q4(q, p.cache, table2, lens2),
                       mq.attention_q4(q, s.cache, s.table, s.lens_t))
    over = buf[:2 * M].view(torch.int32)                    # and under the first row
    over.copy_(s.lens_t)
    for call in (lambda: mq.attention_q4(q, s.cache, table, over, out=out),
                 lambda: mq.kv_store_q4(k, v, s.cache, table, over, freqs=f, q=q, q_out=out),
                 lambda: mq.kv_load_q4(s.cache, table, over, M, k_out=out[:, :2 * D])):
        with pytest.raises(mq.MQError) as e:
            call()
        assert e.value.code == mq._lib.MQ_ERR_OVERLAP


def test_rows_that_see_nothing_and_rows_of_nobody():
    announce("attention_q4 rows that see nothing")
    D, H = 64, 4
    s = filled(D, 2, 32, [40, 40], [40, 40], seed=7)
    q = rows_of(90, H * D, torch.float16, 8)
    out = torch.full_like(q, 5)
    # rows 0 .. 2 and 83 .. 89 belong to no sequence; sequence 0 has 10 tokens for 40 rows
    y = mq.attention_q4(q, s.cache, s.table, ints([10, 40]), cu_rows=ints([3, 43, 83]), out=out)
    assert y is out and bool((out[:3] == 5).all()) and bool((out[83:] == 5).all())
    assert bool((out[3:33] == 0).all()) and not bool((out[33:83] == 0).all(1).any())
    for lens in ([0, 0], [-7, -(1 << 31)]):
        out.fill_(5)
        mq.attention_q4(q[:80], s.cache, s.table, ints(lens), cu_rows=ints([0, 40, 80]), out=out[:80])
        assert bool((out[:80] == 0).all())
    out.fill_(5)                                       # row counts that leave the batch
    mq.attention_q4(q[:80], s.cache, s.table, s.lens_t, cu_rows=ints([-5, 1 << 30, 20]), out=out[:80])
    assert bool((out[80:] == 5).all())
    # a long table, nothing in it: the parts of an empty sequence
    z = mq.attention_q4(q[:1], s.cache, s.table[:1].repeat(1, 3000), ints([0]))
    assert bool((z == 0).all())


def test_bad_pages_are_not_attended_to():
    announce("attention_q4 bad pages")
    D, H, n = 128, 4, 200
    s = filled(D, 2, 32, [1], [n], seed=9, ragged=False)
    q = rows_of(1, H * D, torch.float16, 10)
    qs = to_host(q).astype(np.float64).reshape(1, H, D)
    good = s.table.clone()
    for bad in (-1, s.cache.shape[0], 1 << 30, -(1 << 31)):
        t = good.clone()
        t[0, 1], t[0, 4] = bad, bad
        y = to_host(mq.attention_q4(q, s.cache, t, s.lens_t)).astype(np.float64).reshape(1, H, D)
        keys = [j for j in range(n) if j // 32 not in (1, 4)]
        ref, tol = expect(s, qs, H, 0, [10 ** 6], slice(0, 1), oa.default_scale(D), False, 0, 0.0,
                          None, 0, keys)
        assert (np.abs(y - ref) <= tol).all()
        t.fill_(bad)
        assert bool((mq.attention_q4(q, s.cache, t, s.lens_t) == 0).all())
    # a sequence longer than its table
    y = mq.attention_q4(q, s.cache, good[:, :3].contiguous(), s.lens_t)
    z = mq.attention_q4(q, s.cache, good, ints([96]))
    assert torch.equal(y, z)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_infinities_and_nan_stay_with_the_rows_that_see_them(D):
    announce("attention_q4 special values", D)
    H, Hkv, n = 4, 2, 100
    s = filled(D, Hkv, 32, [n], [n], seed=11, ragged=False)
    q = rows_of(n, H * D, torch.float16, 12)
    clean = mq.attention_q4(q, s.cache, s.table, s.lens_t)
    k, v = (rows_of(1, Hkv * D, torch.float32, i).contiguous() for i in (13, 14))
    for t, which in ((37, "v"), (63, "v"), (64, "k"), (99, "v"), (40, "inf")):
        keep = s.bytes.clone()
        kk, vv = k.clone(), v.clone()
        (kk if which == "k" else vv)[0, D + 5] = float("nan") if which != "inf" else float("inf")
        mq.kv_store_q4(kk, vv, s.cache, s.table, ints([t + 1]))       # head 1 of token t
        y = mq.attention_q4(q, s.cache, s.table, s.lens_t).view(n, H, D)
        c = clean.view(n, H, D)
        assert torch.equal(y[:t], c[:t]), (t, which)
        bad = ~torch.isfinite(y)
        assert not bool(bad[:, :2].any()), (t, which)
        if which == "k":
            assert bool(bad[t:, 2:].all())
        else:                                          # the block of element 5 alone
            assert bool(bad[t:, 2:, :32].all()) and not bool(bad[..., 32:].any())
        w = mq.attention_q4(q, s.cache, s.table, s.lens_t, window=16).view(n, H, D)
        assert bool(torch.isfinite(w[:t]).all()) and bool(torch.isfinite(w[t + 16:]).all())
        assert not bool(torch.isfinite(w[t:t + 16, 2:, :32]).any())
        s.bytes.copy_(keep)
    q2 = q.clone()
    q2[50, 7], q2[51, 2 * D + 1] = float("nan"), float("inf")         # heads 0 and 2
    y = mq.attention_q4(q2, s.cache, s.table, s.lens_t).view(n, H, D)
    bad = ~torch.isfinite(y)
    assert bool(bad[50, 0].all()) and bool(bad[51, 2].all())
    bad[50, 0], bad[51, 2] = False, False
    assert not bool(bad.any())
    same = torch.ones(n, H, dtype=torch.bool, device=dev())
    same[50, 0] = same[51, 2] = False
    assert torch.equal(y[same], clean.view(n, H, D)[same])


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [20, 100])               # few and many rows of a key/value head
def test_blocks_beyond_f16_stay_with_the_rows_that_see_them(D, n):
    """Keys and values that f32 holds and f16 does not: NaN in the rows that see them, in both
    kernels, and no bit changed in the rows before."""
    announce("attention_q4 blocks beyond f16", D, n)
    H, Hkv = 4, 2
    s = filled(D, Hkv, 32, [n], [n], seed=11, ragged=False)
    q = rows_of(n, H * D, torch.float16, 12)
    clean = mq.attention_q4(q, s.cache, s.table, s.lens_t).view(n, H, D)
    k, v = (rows_of(1, Hkv * D, torch.float32, i).contiguous() for i in (13, 14))
    keep = s.bytes.clone()
    for size in (65520.0, -1e5, 524000.0):
        for t in (0, 17, n - 1):
            for which in "kv":
                kk, vv = k.clone(), v.clone()
                (kk if which == "k" else vv)[0, D + 5] = size     # head 1 of token t
                mq.kv_store_q4(kk, vv, s.cache, s.table, ints([t + 1]))
                y = mq.attention_q4(q, s.cache, s.table, s.lens_t).view(n, H, D)
                assert torch.equal(y[:t], clean[:t]), (size, t, which)
                bad = ~torch.isfinite(y)
                assert not bool(bad[:, :2].any())
                if which == "k":
                    assert bool(bad[t:, 2:].all())
                else:
                    assert bool(bad[t:, 2:, :32].all()) and not bool(bad[..., 32:].any())
                s.bytes.copy_(keep)
    # and the largest that are stored: right in both kernels
    kk, vv = k.clone(), v.clone()
    kk[0, D + 5], vv[0, D + 5] = 65519.0, -65519.0
    mq.kv_store_q4(kk, vv, s.cache, s.table, ints([18]))
    lk, lv = mq.kv_load_q4(s.cache, s.table, s.lens_t, n, out_dtype=torch.float32)
    s.k, s.v = (to_host(t).astype(np.float64).reshape(n, Hkv, D) for t in (lk, lv))
    assert abs(s.k[17, 1, 5]) == 65504 and abs(s.v[17, 1, 5]) == 65504
    check(s, H, scale=2.0 ** -16)
    check(s, H, xt="f32", scale=2.0 ** -16, causal=False)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("byte", [0x70, 0xF7, 0x7B, 0xFF])
def test_tokens_never_stored_stay_out_of_rows_that_do_not_see_them(D, byte):
    """Scales of 9088, −30000, 61000 (finite: their products with a code are not) and NaN in
    the bytes behind the tokens that the rows see."""
    announce("attention_q4 tokens never stored", D, byte)
    n, past = 45, 70
    s = filled(D, 1, 32, [n], [n], seed=byte, ragged=False)
    raw = Batch(D, 1, 32, [n + past], [n + past], byte, False)
    raw.bytes.fill_(byte)
    k, v = rows_of(n, D, torch.float16, 100 + byte), rows_of(n, D, torch.float16, 101 + byte)
    mq.kv_store_q4(k, v, raw.cache, raw.table, ints([n]))
    for H, rows in ((1, n + past), (4, n + past), (8, 80)):
        q = rows_of(rows, H * D, torch.float16, 3)
        y = mq.attention_q4(q, raw.cache, raw.table, ints([n + past]))
        at = np.arange(n + past - rows, n)             # positions of the rows before the bytes
        ref, tol = expect(s, to_host(q).astype(np.float64).reshape(rows, H, D), H, 0, at,
                          slice(0, len(at)), oa.default_scale(D), True, 0, 0.0, None, 0)
        got = to_host(y).astype(np.float64).reshape(rows, H, D)[:len(at)]
        assert (np.abs(got - ref) <= tol).all(), (H, rows)


def test_far_pages():
    """A cache past 2^32 bytes."""
    D, Hkv, page = 128, 8, 256
    pages = (9 << 29) // mq.kv_page_bytes(Hkv, page, D) + 2
    announce("attention_q4 far pages", pages)
    cache = torch.empty((pages, Hkv, page // 32, 36 * D), dtype=torch.uint8, device=dev())
    k, v = rows_of(300, Hkv * D, torch.float16, 1), rows_of(300, Hkv * D, torch.float16, 2)
    q = rows_of(300, Hkv * D, torch.float16, 3)
    for m in (1, 7, 300):
        outs = []
        for table in ([[0, 1]], [[pages - 1, pages - 2]]):
            mq.kv_store_q4(k, v, cache, ints(table), ints([300]))
            outs.append(mq.attention_q4(q[:m], cache, ints(table), ints([300])))
        assert torch.equal(outs[0], outs[1])


def test_appending_token_by_token_is_the_prompt():
    """A prompt in one call, in pieces and token by token: each row's result is within
    the two calls' tolerances of the oracle; and rotations, store and attention chained
    between the products of a layer."""
    announce("attention_q4 prompt, pieces, tokens")
    D, H, Hkv, n, hidden = 128, 6, 2, 75, 512
    import synth
    fmt = synth.Q4_K
    N = (H + 2 * Hkv) * D
    g = torch.Generator(device=dev()).manual_seed(4)
    wqkv = torch.from_numpy(synth.weights(fmt, synth.rng(5), N, hidden)).to(dev()).reshape(-1)
    wo = torch.from_numpy(synth.weights(fmt, synth.rng(6), hidden, H * D + (256 - H * D % 256) % 256)
                          ).to(dev()).reshape(-1)
    x = torch.randn(n, hidden, generator=g, device=dev()).half()
    h0 = torch.randn(n, hidden, generator=g, device=dev())
    bias = torch.randn(N, generator=g, device=dev()) * 0.1
    f = mq.rope_freqs(D, device=dev())

    def layer(s, x, h, length):
        qkv = mq.linear_fused(x, wqkv, fmt, N, hidden, bias=bias)
        q, k, v = qkv[:, :H * D], qkv[:, H * D:(H + Hkv) * D], qkv[:, (H + Hkv) * D:]
        q = mq.kv_store_q4(k, v, s.cache, s.table, ints([length]), freqs=f, q=q)
        a = mq.attention_q4(q, s.cache, s.table, ints([length]))
        return q, a, mq.linear_fused(a, wo, fmt, hidden, H * D, residual=h)

    results = []
    for cuts in ([n], [20, 31, 13, 11], [1] * n):
        s = Batch(D, Hkv, 32, [n], [n], 13, False)
        at, parts = 0, []
        for c in cuts:
            parts.append(layer(s, x[at:at + c], h0[at:at + c], at + c))
            at += c
        results.append((s, [torch.cat(p) for p in zip(*parts)]))
    w = mq.dequant_to_f16(wo, fmt, hidden, H * D)[:, :H * D].double()
    for s, (qt, at, yt) in results:
        # (the product's sums may differ with the row count by their last bits, and a
        # piece's cache in a code: each against its own)
        lk, lv = mq.kv_load_q4(s.cache, s.table, s.lens_t, n, out_dtype=torch.float32)
        s.k, s.v = (to_host(t).astype(np.float64).reshape(n, Hkv, D) for t in (lk, lv))
        s.tok = [0, n]
        qs = to_host(qt).astype(np.float64).reshape(n, H, D)
        ref, tol = expect(s, qs, H, 0, np.arange(n), slice(0, n), oa.default_scale(D), True, 0,
                          0.0, None, 0)
        assert (np.abs(to_host(at).astype(np.float64).reshape(n, H, D) - ref) <= tol).all()
        # the o product's own bound, 1e-3 of the sum of magnitudes
        want = h0.double() + at.double() @ w.T
        assert bool(((yt - want).abs() <= 1e-3 * (at.double().abs() @ w.abs().T) + 1e-5).all())


def test_deterministic_on_streams_and_in_graphs():
    announce("attention_q4 streams and graphs")
    D, H, Hkv = 128, 8, 2
    s = filled(D, Hkv, 64, [1, 1, 1], [4000, 900, 33], seed=15, ragged=False)
    q = rows_of(3, H * D, torch.float16, 16)
    y = mq.attention_q4(q, s.cache, s.table, s.lens_t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = mq.attention_q4(q, s.cache, s.table, s.lens_t)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2)
    need = mq.attention_workspace_bytes(s.cache, 3, H, 3, s.table.shape[1] * s.page)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev())
    assert torch.equal(y, mq.attention_q4(q, s.cache, s.table, s.lens_t, ws=ws))
    # two captured calls share the workspace and run one after the other
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    q2 = q * 2
    for g, x, o in zip(graphs, (q, q2), outs):
        with torch.cuda.graph(g):
            mq.attention_q4(x, s.cache, s.table, s.lens_t, out=o, ws=ws)
    for rep in range(4):                               # lengths change under the graphs
        s.lens_t.copy_(ints([4000 - 37 * rep, 900 - 31 * rep, 33 - 11 * rep]))
        want = [mq.attention_q4(x, s.cache, s.table, s.lens_t) for x in (q, q2)]
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(1)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), rep
    del graphs


def test_two_calls_at_once():
    announce("attention_q4 two streams at once")
    a = filled(128, 2, 64, [1, 1], [3000, 2000], seed=17, ragged=False)
    b = filled(64, 4, 32, [30, 50], [400, 50], seed=18)
    qa, qb = rows_of(2, 8 * 128, torch.float16, 19), rows_of(80, 8 * 64, torch.float16, 20)
    ref = (mq.attention_q4(qa, a.cache, a.table, a.lens_t),
           mq.attention_q4(qb, b.cache, b.table, b.lens_t, cu_rows=b.cu))
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            got[0].append(mq.attention_q4(qa, a.cache, a.table, a.lens_t))
        with torch.cuda.stream(streams[1]):
            got[1].append(mq.attention_q4(qb, b.cache, b.table, b.lens_t, cu_rows=b.cu))
    torch.cuda.synchronize()
    for g, r in zip(got, ref):
        assert all(torch.equal(x, r) for x in g)


def test_refusals():
    announce("attention_q4 refusals")
    s = filled(64, 2, 32, [2, 2], [2, 40], seed=21, ragged=False)
    q = rows_of(4, 256, torch.float16, 22)
    base = dict(q=q, cache=s.cache, table=s.table, lens=s.lens_t)
    for kw, text in ((dict(q=q.cpu()), "GPU tensor"), (dict(q=q.double()), "float32 or float16"),
                     (dict(q=q[0]), "2-D"), (dict(q=q.t()), "unit column stride"),
                     (dict(q=q[:, :100]), "multiple of head_dim"), (dict(cache=s.cache.cpu()), "same GPU"),
                     (dict(cache=s.bytes), "cache must be"), (dict(table=s.table.float()), "torch.int32"),
                     (dict(lens=s.lens_t[:1]), "lens must be"), (dict(cu_rows=ints([0, 4])), "cu_rows must"),
                     (dict(slopes=torch.ones(3, device=dev())), "slopes must be"),
                     (dict(slopes=torch.ones(4, device=dev()).half()), "slopes must be"),
                     (dict(slopes=torch.ones(4)), "same GPU"), (dict(prefix=ints([1])), "prefix must be"),
                     (dict(prefix=s.lens_t.long()), "prefix must be"),
                     (dict(out=q.float()), "out must be torch.float16"), (dict(out=q[:3]), "out must be"),
                     (dict(out=q.cpu()), "same GPU"), (dict(ws=torch.zeros(9)), "ws must be")):
        with pytest.raises(ValueError, match=text):
            mq.attention_q4(**{**base, **kw})
    for kw, code in ((dict(q=q[:0]), "SHAPE"), (dict(q=q[:3]), "SHAPE"), (dict(q=q[:, :192]), "SHAPE"),
                     (dict(window=-1), "EPS"), (dict(cap=-1.0), "EPS"), (dict(cap=1e300), "EPS"),
                     (dict(scale=float("nan")), "EPS"), (dict(max_len=-1), "SHAPE"), (dict(out=q), "OVERLAP"),
                     (dict(max_len=1 << 20, ws=torch.empty(16, dtype=torch.uint8, device=dev())), "WORKSPACE")):
        with pytest.raises(mq.MQError) as e:
            mq.attention_q4(**{**base, **kw})
        assert e.value.code == getattr(mq._lib, "MQ_ERR_" + code), kw
    for kw in (dict(scale="x"), dict(cap=None), dict(window=1.5)):
        with pytest.raises(TypeError):
            mq.attention_q4(**{**base, **kw})
    with pytest.raises(OverflowError):
        mq.attention_q4(**base, max_len=1 << 70)
