"""Linear layers with their epilogue, and gated ones, against the f64 oracle.

Tolerances, with u = 2^-24 and S = |X|·|W|ᵀ + |bias| per element:
  * the sums: products of f16 values are exact in f32; a sum runs through at
    most K/16 accumulations of 16 products, 16 more joins of K ranges and the
    bias: dv = (K/16 + 48)·u·S;
  * the activations: |act'| <= 1.13, so dv costs at most 1.13·dv.  Their own
    evaluation: exp, reciprocal and products are within 12·u; silu's and
    gelu_tanh's exponent t is off by at most 4·u·|t|, which is the relative
    error of e^-t, with |t| <= 1.6·|v| + 0.08·|v|³; gelu's erfc argument is off
    by 2·u of itself, which moves erfc by at most 2·u·v² (+ v² for the square);
    together da = (12 + 8·|v| + 4·v² + |v|³)·u·|act(v)|;
  * residual, product with the up sums and the sum of both: one rounding each;
  * the output type: half a step, 2^-24 (f32) or 2^-11 (f16, 2^-25 below its
    smallest normal) of the value; from 65504 + half a step = 65520 on an f16
    output is infinite, by the definition of rounding to nearest.
"""

import numpy as np
import pytest

import oracle
import synth
from gpu_common import announce, dev, needs_gpu, to_dev_f16, to_dev_u8, to_host
from oracle import layers

pytestmark = [pytest.mark.gpu, needs_gpu]

import torch  # noqa: E402

import quantized_weight_prefill_q4_amd as mq  # noqa: E402
from quantized_weight_prefill_q4_amd import _lib  # noqa: E402

U = 2.0 ** -24
T = {"f32": torch.float32, "f16": torch.float16}
FMTS = [synth.Q4_0, synth.Q5_0, synth.Q5_1, synth.Q8_0, synth.Q4_K, synth.Q5_K, synth.Q6_K]
ACTS = list(layers.ACTS)


def _dv(K, S):
    return (K / 16 + 48) * U * S


def _da(v, act):
    a = np.abs(v)
    rel = 0 if act in ("none", "relu") else 12 + 8 * a + 4 * a * a + a ** 3
    return rel * U * np.abs(layers.act_ref(v, act)) + 1e-36


def _out(y, err, yt):
    if yt == "f32":
        return err * (1 + U) + U * np.abs(y) + 1e-44
    return err * (1 + 2.0 ** -11) + 2.0 ** -11 * np.abs(y) + 2.0 ** -25


def _worst(got, y, tol, yt):
    """The largest error in units of its tolerance."""
    got = to_host(got).astype(np.float64)
    with np.errstate(invalid="ignore"):
        ratio = np.abs(got - y) / tol
    if yt == "f16":
        ratio[np.isinf(got) & (np.sign(got) == np.sign(y)) & (np.abs(y) + tol >= 65520)] = 0
    return np.max(ratio)


def _weight(fmt, rows, K, seed):
    """(the library's weight tensor, f16 bits of its values); fmt 0: the f16 cache."""
    if fmt == 0:
        bits = synth.activations(synth.rng(40, seed), rows, K)
        scaled = (bits.view(np.float16) * np.float16(0.05)).astype(np.float16).view(np.uint16)
        ld = mq.cache_ld(K)
        buf = torch.full((rows, ld), float("nan"), dtype=torch.float16, device=dev())
        buf[:, :K] = to_dev_f16(scaled)
        return buf, scaled
    q = synth.weights(fmt, synth.rng(41, seed, fmt, rows), rows, K)
    return to_dev_u8(q), oracle.dequant_ref(fmt, q, rows, K)


def _x(M, K, xt, seed):
    """(x on the device, its f16 bits): f32 activations are rounded to f16."""
    if xt == "f16":
        bits = synth.activations(synth.rng(42, seed), M, K)
        return to_dev_f16(bits), bits
    x = np.random.default_rng([43, seed]).standard_normal((M, K)).astype(np.float32)
    return torch.from_numpy(x).to(dev()), oracle.activations_to_f16(x)


def _vec(shape, seed, scale=1.0):
    return (scale * np.random.default_rng([44, seed]).standard_normal(shape)).astype(np.float32)


def _guarded(M, N, yt, pad):
    buf = torch.full((M, N + pad), float("nan"), dtype=T[yt], device=dev())
    return buf, buf[:, :N]


def _untouched(buf, M, N):
    return bool(torch.isnan(buf[:, N:]).all())


def check_linear(fmt, M, N, K, xt="f16", bias=True, act="none", rt="f32", yt="f32", split=0, pad=3,
                 seed=0):
    announce("linear", f"fmt={fmt}", M, N, K, xt, f"bias={bias}", act, rt, yt, f"split={split}")
    w, wb = _weight(fmt, N, K, seed)
    x, xb = _x(M, K, xt, seed)
    b = _vec(N, seed) if bias else None
    r = None if rt is None else _vec((M, N), seed + 1, 3.0).astype(np.float16 if rt == "f16"
                                                                   else np.float32)
    v, S = oracle.gemm_ref(xb, wb, K)
    if bias:
        v, S = v + b.astype(np.float64), S + np.abs(b)
    y = layers.act_ref(v, act)
    err = 1.13 * _dv(K, S) + _da(v, act)
    if r is not None:
        y = y + r.astype(np.float64)
        err = err + U * (np.abs(y) + err)
    tol = _out(y, err, yt)
    bd = None if b is None else torch.from_numpy(b).to(dev())
    rd = None
    if r is not None:
        rd = torch.full((M, N + pad + 2), float("nan"), dtype=T[rt], device=dev())[:, :N]
        rd.copy_(torch.from_numpy(r))
    buf, out = _guarded(M, N, yt, pad)
    kw = dict(bias=bd, act=act, residual=rd, split_k=split)
    if fmt == 0:
        got = mq.linear_f16cache(x, w, K, out=out, **kw)
        again = mq.linear_f16cache(x, w, K, out_dtype=T[yt], **kw)
    else:
        got = mq.linear_fused(x, w, fmt, N, K, out=out, **kw)
        again = mq.linear_fused(x, w, fmt, N, K, out_dtype=T[yt], **kw)
    assert got is out
    worst = _worst(got, y, tol, yt)
    assert worst <= 1, f"{worst:.3g} times the tolerance"
    assert torch.equal(got, again) and _untouched(buf, M, N)
    return worst


def check_glu(fmt, M, N, K, xt="f16", bias=True, act="silu", yt="f16", split=0, pad=3, seed=0):
    announce("glu", f"fmt={fmt}", M, N, K, xt, f"bias={bias}", act, yt, f"split={split}")
    w, wb = _weight(fmt, 2 * N, K, seed)
    x, xb = _x(M, K, xt, seed)
    b = _vec(2 * N, seed) if bias else None
    y, g, u, Sg, Su = layers.glu_ref(xb, wb, K, b, act)
    a = layers.act_ref(g, act)
    eg, eu = 1.13 * _dv(K, Sg) + _da(g, act), _dv(K, Su)
    err = eg * np.abs(u) + np.abs(a) * eu + eg * eu
    tol = _out(y, err + U * (np.abs(y) + err), yt)
    bd = None if b is None else torch.from_numpy(b).to(dev())
    buf, out = _guarded(M, N, yt, pad)
    kw = dict(bias=bd, act=act, split_k=split)
    if fmt == 0:
        got = mq.glu_f16cache(x, w, K, out=out, **kw)
        again = mq.glu_f16cache(x, w, K, out_dtype=T[yt], **kw)
    else:
        got = mq.glu_fused(x, w, fmt, N, K, out=out, **kw)
        again = mq.glu_fused(x, w, fmt, N, K, out_dtype=T[yt], **kw)
    assert got is out
    worst = _worst(got, y, tol, yt)
    assert worst <= 1, f"{worst:.3g} times the tolerance"
    assert torch.equal(got, again) and _untouched(buf, M, N)
    return worst


# sizes: few rows, a row tile and one more, ragged and odd columns, wide outputs
# that take 256 x 256 tiles (more than 192 of them), long K split over the tail
SHAPES = [(1, 64, 256), (1, 1, 512), (2, 333, 512), (5, 130, 1024), (8, 1000, 768),
          (13, 257, 2048), (16, 96, 512), (17, 100, 256),
          (24, 33, 4096), (31, 8209, 256), (32, 515, 1280), (33, 515, 512), (64, 128, 512),
          (65, 129, 256), (100, 300, 1024), (128, 256, 512), (200, 520, 768), (257, 1001, 512),
          (300, 640, 4096)]


@pytest.mark.parametrize("fmt", [0] + FMTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_shapes(fmt, shape):
    i = SHAPES.index(shape) + FMTS.index(fmt) if fmt else SHAPES.index(shape)
    check_linear(fmt, *shape, xt=("f16", "f32")[i % 2], act=ACTS[i % 5], bias=i % 3 != 0,
                 rt=(None, "f32", "f16")[(i // 2) % 3], yt=("f32", "f16")[(i // 3) % 2], seed=i)


@pytest.mark.parametrize("fmt", [0] + FMTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_glu_shapes(fmt, shape):
    i = SHAPES.index(shape) + FMTS.index(fmt) if fmt else SHAPES.index(shape)
    check_glu(fmt, *shape, xt=("f16", "f32")[i % 2], act=ACTS[(i + 2) % 5], bias=i % 2 == 0,
              yt=("f32", "f16")[(i // 2) % 2], seed=i)


@pytest.mark.parametrize("fmt", [0, synth.Q4_0, synth.Q5_0, synth.Q5_1, synth.Q8_0])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 288, 1056, 2016])
def test_part_units(fmt, K):
    """Rows that end inside a unit of 256 and inside a lane's pair of blocks;
    the last weight row's end is the buffer's."""
    for M in (1, 4, 5, 16, 17, 32):
        check_linear(fmt, M, 47, K, act="silu", rt="f32", yt="f32", seed=K)
        check_glu(fmt, M, 31, K, yt="f32", seed=K)
    if fmt == 0:
        check_linear(fmt, 3, 47, K - 24, yt="f32", seed=K)      # 8 halves
        check_linear(fmt, 9, 33, K + 8, xt="f32", yt="f32", seed=K)


@pytest.mark.parametrize("fmt", [0] + FMTS)
def test_long_rows(fmt):
    """As many waves per workgroup as each number of rows can have (K of 16
    units and more), their LDS up to the compute unit's; and one tile too few
    or too many for a round of the chip."""
    for M in (2, 8, 16, 31):
        check_linear(fmt, M, 40, 5120, act="silu", rt="f32", yt="f32", seed=M)
        check_glu(fmt, M, 33, 4096, xt="f32", yt="f32", seed=M)
    check_linear(fmt, 3, 4128, 1024, rt="f16", yt="f16")
    check_glu(fmt, 9, 2064, 768, yt="f16")


def test_one_row_of_a_wider_buffer():
    """The stride of a single row is of no account."""
    K, N = 256, 48
    announce("single row, any stride")
    w, _ = _weight(0, N, K, 31)
    x, _ = _x(3, K, "f16", 31)
    buf = torch.zeros(3, K + 8, dtype=torch.float16, device=dev())
    buf[:, :K] = x
    odd = buf.view(-1)[:3 * (K + 8)].as_strided((1, K), (K + 3, 1))
    assert torch.equal(mq.linear_f16cache(odd, w, K), mq.linear_f16cache(x[:1], w, K))
    out = torch.zeros(1, N + 5, device=dev())
    mq.linear_f16cache(x[:1], w, K, out=out[:, :N].as_strided((1, N), (3, 1)))
    assert torch.equal(out[:, :N], mq.linear_f16cache(x[:1], w, K))
    assert torch.equal(mq.glu_f16cache(odd, w, K), mq.glu_f16cache(x[:1], w, K))


@pytest.mark.parametrize("fmt", FMTS)
def test_few_rows_see_the_cache_weights(fmt):
    """One-hot activations read every weight back: the few-row kernels expand
    the values of the f16 cache (an exact zero's sign aside)."""
    N, K = 50, 512
    announce("one-hot", fmt)
    q, bits = _weight(fmt, N, K, 30)
    want = torch.from_numpy(bits.view(np.float16).astype(np.float32)).to(dev())
    eye = torch.eye(K, dtype=torch.float16, device=dev())
    got = torch.cat([mq.linear_fused(eye[k:k + 16], q, fmt, N, K) for k in range(0, K, 16)])
    assert torch.equal(got.t(), want)
    got = torch.cat([mq.linear_fused(eye[k:k + 3].float(), q, fmt, N, K) for k in range(0, K, 3)])
    assert torch.equal(got.t(), want)
    got = torch.cat([mq.linear_fused(eye[k:k + 32], q, fmt, N, K) for k in range(0, K, 32)])
    assert torch.equal(got.t(), want)


@pytest.mark.parametrize("fmt", [synth.Q4_0, synth.Q5_0, synth.Q5_1, synth.Q8_0])
def test_few_rows_see_extreme_scales(fmt):
    """The same with block scales from the smallest subnormal to the largest
    whose products stay finite, of both signs, and zero: what is expanded in f16
    arithmetic rounds as the cache's values do, subnormal results included."""
    N, K = 40, 256
    announce("one-hot, extreme scales", fmt)
    q = synth.weights(fmt, synth.rng(48, fmt), N, K).copy()
    blocks = q.reshape(-1, mq.block_bytes(fmt))
    scales = np.array([0x0001, 0x0003, 0x00FF, 0x03FF, 0x0400, 0x0401, 0x07FF, 0x1234, 0x3555,
                       0x3C01, 0x4FFF, 0x5FFE, 0x8001, 0x83FF, 0x8401, 0xB7FD, 0xDFFE, 0x0000,
                       0x8000], np.uint16)
    blocks[:, :2] = scales[np.arange(len(blocks)) % len(scales)].view(np.uint8).reshape(-1, 2)
    want = oracle.dequant_ref(fmt, q, N, K).view(np.float16).astype(np.float32)
    assert np.isfinite(want).all()
    w = to_dev_u8(q)
    eye = torch.eye(K, dtype=torch.float16, device=dev())
    for rows in (4, 16, 32):
        got = torch.cat([mq.linear_fused(eye[k:k + rows], w, fmt, N, K)
                         for k in range(0, K, rows)])
        assert np.array_equal(got.t().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", [0, synth.Q6_K, synth.Q8_0])
def test_several_tiles_per_compute_unit(fmt):
    """Two, three and four workgroups to a compute unit, whose numbers of waves
    differ with the rows, their type and the layer."""
    for N in (4200, 8300, 12400):
        check_glu(fmt, 6, N, 1024, xt="f32", yt="f16", seed=N)
        check_linear(fmt, 13, N, 1024, rt="f16", yt="f32", seed=N)
    check_glu(fmt, 2, 12400, 2048, yt="f32")


@pytest.mark.parametrize("fmt", [0] + FMTS)
def test_wide_outputs(fmt):
    """256 x 256 tiles, the last ones ragged in rows and columns."""
    N, K = 24903, 256 if fmt != synth.Q8_0 else 288     # 288: not a multiple of 256
    p = mq.gemm_plan(fmt, 300, N, K)
    assert (p["bm"], p["bn"]) == (256, 256)
    check_linear(fmt, 300, N, K, act="silu", rt="f16", yt="f32")
    check_glu(fmt, 300, N // 2, K, yt="f16")
    if fmt == synth.Q8_0:
        check_linear(fmt, 300, N, 256, act="gelu", rt="f32", yt="f16")
        check_glu(fmt, 300, N // 2 + 1, 256, act="gelu_tanh", yt="f32")


@pytest.mark.parametrize("fmt", [0, synth.Q4_K, synth.Q6_K, synth.Q8_0, synth.Q5_1])
@pytest.mark.parametrize("split", [1, 2, 3, 5, 8, 16])
def test_forced_splits(fmt, split):
    check_linear(fmt, 70, 333, 2048, split=split, act="gelu_tanh", rt="f16", yt="f16", seed=split)
    check_glu(fmt, 150, 161, 2048, split=split, yt="f32", seed=split)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("yt", ["f32", "f16"])
def test_every_epilogue(act, yt):
    for M in (3, 40, 300):
        for rt in (None, "f32", "f16"):
            for bias in (False, True):
                check_linear(0, M, 136, 264, act=act, rt=rt, yt=yt, bias=bias, pad=5)
        check_glu(0, M, 68, 264, act=act, yt=yt)


@pytest.mark.parametrize("M", [1, 3, 40, 100, 300, 1100])
@pytest.mark.parametrize("fmt", [0, synth.Q4_K])
def test_sums_are_the_products(fmt, M):
    """Without an epilogue and unsplit the tile kernels' f32 sums are the GEMM's
    bit for bit; the few-row kernels' order differs."""
    N, K = 520, 1024
    w, _ = _weight(fmt, N, K, 5)
    x, _ = _x(M, K, "f16", 5)
    announce("linear == gemm", fmt, M)
    if fmt == 0:
        a, b = mq.linear_f16cache(x, w, K, split_k=1), mq.gemm_f16cache(x, w, K, split_k=1)
    else:
        a = mq.linear_fused(x, w, fmt, N, K, split_k=1)
        b = mq.gemm_fused(x, w, fmt, N, K, split_k=1)
    if M > 64:
        assert torch.equal(a, b)
    else:
        xa = x.double().abs() @ (w[:, :K].double().abs().t() if fmt == 0 else
                                 mq.dequant_to_f16(w, fmt, N, K)[:, :K].double().abs().t())
        assert bool(((a.double() - b.double()).abs() <= 2 * (K / 16 + 48) * U * xa).all())


@pytest.mark.parametrize("M", [1, 40, 300])
def test_in_place_residual_and_special_values(M):
    """The residual stream updated in place; NaN and infinities in one row of x
    stay in that row of y; a saturating sum rounds to an f16 infinity."""
    N, K = 200, 512
    w, _ = _weight(0, N, K, 6)
    x, _ = _x(M, K, "f16", 6)
    announce("linear in place", M)
    r = torch.from_numpy(_vec((M, N), 6)).to(dev())
    want = mq.linear_f16cache(x, w, K, act="silu", residual=r)
    s = r.clone()
    assert mq.linear_f16cache(x, w, K, act="silu", residual=s, out=s) is s
    assert torch.equal(s, want)
    s16 = r.half()
    want16 = mq.linear_f16cache(x, w, K, residual=s16.clone(), out_dtype=torch.float16)
    mq.linear_f16cache(x, w, K, residual=s16, out=s16)
    assert torch.equal(s16, want16)
    if M > 2:
        bad = x.clone()
        bad[1, 7], bad[2, 9] = float("nan"), float("inf")
        y = mq.linear_f16cache(bad, w, K, act="silu", residual=r)
        keep = [i for i in range(M) if i not in (1, 2)]
        assert torch.equal(y[keep], want[keep]) and bool(torch.isnan(y[1]).all())
        g = mq.glu_f16cache(bad, w, K)
        assert torch.equal(g[keep], mq.glu_f16cache(x, w, K)[keep])
        assert bool(torch.isnan(g[1]).all())
    big = torch.full((M, K), 1000.0, dtype=torch.float16, device=dev())
    ones = torch.ones(N, K, dtype=torch.float16, device=dev())
    y = mq.linear_f16cache(big, ones, K, out_dtype=torch.float16)
    assert bool(torch.isinf(y).all()) and bool((y > 0).all())
    y = mq.linear_f16cache(-big, ones, K, act="silu")
    assert bool((y == 0).all())                     # −512000·e^−512000


def test_strided_activations():
    """Rows of a wider buffer (x, the cache's slices, the outputs of two layers
    side by side) and a converted f32 view."""
    M, N, K = 40, 96, 256
    announce("strided linear")
    w, _ = _weight(0, 2 * N, K, 8)
    wide = torch.full((M, K + 64), float("nan"), dtype=torch.float16, device=dev())
    x, _ = _x(M, K, "f16", 8)
    wide[:, 8:8 + K] = x
    want = mq.linear_f16cache(x, w[:N], K)
    assert torch.equal(mq.linear_f16cache(wide[:, 8:8 + K], w[:N], K), want)
    x32 = torch.full((M, K + 12), float("nan"), device=dev())
    x32[:, 4:4 + K] = x.float()
    assert torch.equal(mq.linear_f16cache(x32[:, 4:4 + K], w[:N], K), want)
    both = torch.empty(M, 2 * N, device=dev())
    mq.linear_f16cache(x, w[:N], K, out=both[:, :N])
    mq.linear_f16cache(x, w[N:], K, out=both[:, N:])
    assert torch.equal(both[:, :N], want)
    assert torch.equal(both[:, N:], mq.linear_f16cache(x, w[N:], K))


def test_layers_replay_in_a_graph():
    """Every layer with and without a K split, captured once and replayed with
    new inputs, against the eager calls; two graphs with a workspace each."""
    K, N = 2048, 320
    announce("layers in a graph")
    wc, _ = _weight(0, N, K, 9)
    wq, _ = _weight(synth.Q4_K, N, K, 9)
    calls = []
    for M, xt in ((1, "f16"), (5, "f32"), (100, "f16"), (300, "f32")):
        x, _ = _x(M, K, xt, M)
        r = torch.from_numpy(_vec((M, N), M)).to(dev())
        for fmt, w in ((0, wc), (synth.Q4_K, wq)):
            for glu in (False, True):
                n = N // 2 if glu else N
                nb = mq.linear_workspace_bytes(fmt, M, n, K, x_f32=xt == "f32", glu=glu)
                ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=dev())

                def call(out=None, ws=None, x=x, r=r, fmt=fmt, w=w, glu=glu, n=n):
                    kw = dict(act="silu", out=out, ws=ws)
                    if fmt and glu:
                        return mq.glu_fused(x, w, fmt, n, K, **kw)
                    if fmt:
                        return mq.linear_fused(x, w, fmt, n, K, residual=r, **kw)
                    if glu:
                        return mq.glu_f16cache(x, w, K, **kw)
                    return mq.linear_f16cache(x, w, K, residual=r, **kw)

                calls.append((call, call(), ws, x))
    outs = [torch.empty_like(y) for _, y, _, _ in calls]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for (call, y, ws, _), o in zip(calls, outs):
            call(out=o, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    for (_, y, _, _), o in zip(calls, outs):
        assert torch.equal(y, o)                    # another stream, same result
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for k, g in enumerate(graphs):
        with torch.cuda.graph(g):
            for (call, _, ws, _), o in list(zip(calls, outs))[k::2]:
                call(out=o, ws=ws)
    xs = {id(x): x for _, _, _, x in calls}
    for rep in range(3):
        for o in outs:
            o.fill_(float("nan"))
        for x in xs.values():
            x.mul_(0.5)
        want = [call() for call, _, _, _ in calls]
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, (o, w) in enumerate(zip(outs, want)):
            assert torch.equal(o, w), f"replay {rep}, call {i}"
    del graphs


def test_two_streams_at_once():
    """Two calls that overlap in time, each with a workspace of its own."""
    M, N, K = 300, 512, 8192
    w, _ = _weight(0, N, K, 10)
    xs = [_x(M, K, "f32", i)[0] for i in (1, 2)]
    announce("two streams")
    want = [mq.linear_f16cache(x, w, K, act="gelu") for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(mq.linear_f16cache(x, w, K, act="gelu"))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


def test_a_feed_forward_block():
    """The operators together, as a layer runs them: the residual norm, the
    gated pair and the down projection onto the stream, on both weight paths
    and for one token as for many; against the f64 composition."""
    H, F = 512, 768
    fmt_gu, fmt_d = synth.Q4_K, synth.Q6_K
    qgu, wgu = _weight(fmt_gu, 2 * F, H, 11)
    qd, wd = _weight(fmt_d, H, F, 12)
    cgu = mq.dequant_to_f16(qgu, fmt_gu, 2 * F, H)
    cd = mq.dequant_to_f16(qd, fmt_d, H, F)
    nw = torch.from_numpy(1 + _vec(H, 13, 0.2)).to(dev())
    for M in (1, 7, 130):
        announce("feed-forward block", M)
        x = torch.from_numpy(_vec((M, H), 14)).to(dev())
        stream = torch.from_numpy(_vec((M, H), 15, 2.0)).to(dev())
        y, h = mq.add_rms_norm(x, nw, residual=stream)
        a = mq.glu_fused(y, qgu, fmt_gu, F, H)
        out = mq.linear_fused(a, qd, fmt_d, H, F, residual=h)
        a2 = mq.glu_f16cache(y, cgu, H)
        out2 = mq.linear_f16cache(a2, cd, F, residual=h)
        # step by step, each from the f16 activations the step before gave
        ry, rh = layers.rms_norm_ref(to_host(x), to_host(nw), 1e-6, to_host(stream))
        assert np.max(np.abs(to_host(y) - ry) / (2.0 ** -11 * np.abs(ry) + 1e-5)) <= 1.01
        yb = to_host(y).view(np.uint16)
        ra, g, u, Sg, Su = layers.glu_ref(yb, wgu, H)
        eg = 1.13 * _dv(H, Sg) + _da(g, "silu")
        err = eg * np.abs(u) + np.abs(layers.act_ref(g, "silu")) * _dv(H, Su)
        for av in (a, a2):
            assert _worst(av, ra, _out(ra, 1.01 * err, "f16"), "f16") <= 1
        for av, ov in ((a, out), (a2, out2)):
            # an activation that f16 cannot hold is infinite, and so (or NaN, where
            # it meets a zero weight or another infinity) is its whole output row
            ah, oh = to_host(av), to_host(ov)
            fine = np.isfinite(ah).all(axis=1)
            assert fine.any() and not np.isfinite(oh[~fine]).any()
            ro, S = layers.linear_ref(ah[fine].view(np.uint16), wd, F, residual=rh[fine])
            e = _dv(F, S)
            assert np.all(np.abs(oh[fine] - ro) <= e + 2 * U * (np.abs(ro) + e))


def test_far_rows():
    """Weights whose halves lie more than 2 GiB apart, and outputs past 2^31
    elements' offsets."""
    K, N = 16384, 66000
    announce("glu far rows")
    w = torch.zeros(2 * N, K, dtype=torch.float16, device=dev())
    w[N - 1, :] = 1.0
    w[2 * N - 1, :] = 2.0
    w[N // 2, 5] = 3.0
    w[N + N // 2, 6] = 4.0
    for M in (1, 3, 200):
        x = torch.zeros(M, K, dtype=torch.float16, device=dev())
        x[:, 5:7] = 1.0
        y = mq.glu_f16cache(x, w, K, act="none", out_dtype=torch.float32)
        assert bool((y[:, N - 1] == 2 * 4).all()) and bool((y[:, N // 2] == 12).all())
        assert int((y != 0).sum()) == 2 * M
    del w, y
    torch.cuda.empty_cache()


def test_far_quantized_rows():
    """A gated layer whose quantized weight passes 2 GiB, few rows and many."""
    K, N = 16384, 62000
    announce("glu far quantized rows")
    row = mq.row_bytes("q8_0", K)
    assert 2 * N * row > 1 << 31
    q = torch.zeros(2 * N, K // 32, 34, dtype=torch.uint8, device=dev())
    one = torch.tensor([1.0], dtype=torch.float16, device=dev()).view(torch.uint8)
    q[..., 0:2] = one
    q[N - 1, 0, 2 + 5] = 1
    q[2 * N - 1, 0, 2 + 6] = 2
    q[N // 2, 0, 2 + 5] = 3
    q[N + N // 2, 0, 2 + 6] = 4
    for M in (1, 40, 200, 300):
        x = torch.zeros(M, K, dtype=torch.float16, device=dev())
        x[:, 5:7] = 1.0
        y = mq.glu_fused(x, q.view(-1), "q8_0", N, K, act="none", out_dtype=torch.float32)
        assert bool((y[:, N - 1] == 2).all()) and bool((y[:, N // 2] == 12).all()), M
        assert int((y != 0).sum()) == 2 * M
    del q, y
    torch.cuda.empty_cache()


def test_binding_refuses():
    M, N, K = 4, 64, 256
    announce("linear refusals")
    w, _ = _weight(0, N, K, 20)
    q, _ = _weight(synth.Q4_K, N, K, 20)
    x, _ = _x(M, K, "f16", 20)
    b = torch.zeros(N, device=dev())
    r = torch.zeros(M, N, device=dev())
    ok = dict(x=x, w16=w, K=K, bias=b, residual=r)
    for kw, text in ((dict(x=x.cpu()), "GPU tensor"), (dict(x=x.double()), "float32 or float16"),
                     (dict(x=x[0]), "2-D"), (dict(x=x[:, :K - 8]), "x must be at least"),
                     (dict(x=x.t()), "unit column"), (dict(w16=w.float()), "w16 must be"),
                     (dict(w16=w.cpu()), "same GPU"), (dict(w16=w[:, :K - 8]), "w16 must be at"),
                     (dict(bias=b[:-1]), "contiguous vector"), (dict(bias=b.half()), "float32"),
                     (dict(act="swish"), "unknown activation"),
                     (dict(residual=r[:, :-1]), "residual must be at least"),
                     (dict(residual=r[:-1]), "residual must be at least"),
                     (dict(residual=r.bfloat16()), "float32 or float16"),
                     (dict(out_dtype=torch.int8), "out_dtype"),
                     (dict(out=r[:, :-1]), "out must be at least"),
                     (dict(ws=torch.empty(64, 2, device=dev())[:, 0]), "ws must be contiguous")):
        with pytest.raises(ValueError, match=text):
            mq.linear_f16cache(**{**ok, **kw})
    for kw, code in ((dict(residual=r[:1].expand(M, N)), _lib.MQ_ERR_LD),
                     (dict(residual=r[:, 1:], w16=w[:-1], bias=None, out=r[:, :-1]),
                      _lib.MQ_ERR_OVERLAP),
                     (dict(K=100), _lib.MQ_ERR_SHAPE), (dict(x=x[:0]), _lib.MQ_ERR_SHAPE),
                     (dict(split_k=17), _lib.MQ_ERR_SPLIT),
                     (dict(split_k=4, ws=torch.empty(8, dtype=torch.uint8, device=dev())),
                      _lib.MQ_ERR_WORKSPACE)):
        with pytest.raises(mq.MQError) as e:
            mq.linear_f16cache(**{**ok, **kw})
        assert e.value.code == code, kw
    with pytest.raises(ValueError, match="wq holds"):
        mq.linear_fused(x, q[:-1], "q4_k", N, K)
    with pytest.raises(ValueError, match="wq holds"):
        mq.glu_fused(x, q, "q4_k", N, K)
    with pytest.raises(ValueError, match="even number"):
        mq.glu_f16cache(x, w[:-1], K)
    with pytest.raises(ValueError, match="contiguous vector"):
        mq.glu_f16cache(x, w, K, bias=b[:N // 2])
    assert mq.glu_fused(x, q, "q4_k", N // 2, K).shape == (M, N // 2)


def test_strides_beyond_int_are_refused():
    """Rows 2^31 elements apart, in every place a layer or a norm takes rows."""
    K = N = 64
    announce("strides beyond int")
    buf = torch.empty((1 << 31) + 64, dtype=torch.float16, device=dev())
    far = buf.as_strided((2, K), (1 << 31, 1))
    x, r = torch.zeros(2, K, dtype=torch.float16, device=dev()), torch.zeros(2, N, device=dev())
    w = torch.zeros(N, K, dtype=torch.float16, device=dev())
    far_w = buf.as_strided((2, K), (1 << 31, 1))
    q = torch.zeros(N * mq.row_bytes("q8_0", K), dtype=torch.uint8, device=dev())
    ones = torch.ones(K, device=dev())
    for call in (lambda: mq.linear_f16cache(far, w), lambda: mq.linear_f16cache(x, far_w),
                 lambda: mq.linear_f16cache(x, w, residual=far),
                 lambda: mq.linear_f16cache(x, w, out=far),
                 lambda: mq.linear_fused(x, q, "q8_0", N, residual=far, out=far),
                 lambda: mq.glu_f16cache(far, w), lambda: mq.glu_f16cache(x, w, out=far),
                 lambda: mq.glu_fused(x, q, "q8_0", N // 2, out=far),
                 lambda: mq.add_rms_norm(far, ones), lambda: mq.add_rms_norm(x, ones, out=far),
                 lambda: mq.add_rms_norm(x, ones, residual=far, residual_out=far),
                 lambda: mq.add_rms_norm(x, ones, residual=r.half(), residual_out=far),
                 lambda: mq.add_rms_norm_q8_1(far, ones)):
        with pytest.raises(ValueError, match="elements apart"):
            call()
    # one row of such a view has no stride
    y = mq.linear_f16cache(x[:1], w, residual=r[:1], out=far[1:])
    assert y.shape == (1, N) and bool((y == 0).all())
    del buf, far, far_w
    torch.cuda.empty_cache()


@pytest.mark.parametrize("K", [0, -1, -64])
def test_sizes_below_one_are_refused(K):
    """A K (or an N of block weights) that is not a size is refused, as the GEMM
    entry points do; None alone stands for the activations' width."""
    announce("K below one", K)
    x = torch.zeros(3, 64, dtype=torch.float16, device=dev())
    w = torch.zeros(32, 64, dtype=torch.float16, device=dev())
    q = torch.zeros(32 * mq.row_bytes("q8_0", 64), dtype=torch.uint8, device=dev())
    for call in (lambda: mq.linear_f16cache(x, w, K), lambda: mq.glu_f16cache(x, w, K),
                 lambda: mq.linear_fused(x, q, "q8_0", 32, K),
                 lambda: mq.glu_fused(x, q, "q8_0", 16, K),
                 lambda: mq.linear_fused(x, q, "q8_0", K, 64),
                 lambda: mq.glu_fused(x, q, "q8_0", K, 64), lambda: mq.gemm_f16cache(x, w, K)):
        with pytest.raises(mq.MQError) as e:
            call()
        assert e.value.code == _lib.MQ_ERR_SHAPE
    assert mq.linear_f16cache(x, w, None).shape == (3, 32)


def test_vectors_of_another_size_are_refused():
    """A bias or a norm's weights that are longer than the layer's are another
    layer's."""
    K, N = 64, 32
    announce("longer vectors")
    x = torch.zeros(3, K, dtype=torch.float16, device=dev())
    w = torch.zeros(N, K, dtype=torch.float16, device=dev())
    q = torch.zeros(N * mq.row_bytes("q8_0", K), dtype=torch.uint8, device=dev())
    v = torch.ones(K + 1, device=dev())
    for n in (N + 1, K):
        for call in (lambda: mq.linear_f16cache(x, w, bias=v[:n]),
                     lambda: mq.linear_fused(x, q, "q8_0", N, bias=v[:n]),
                     lambda: mq.glu_f16cache(x, w, bias=v[:n]),
                     lambda: mq.glu_fused(x, q, "q8_0", N // 2, bias=v[:n])):
            with pytest.raises(ValueError, match=f"contiguous vector of {N} elements"):
                call()
    for call in (mq.add_rms_norm, mq.add_rms_norm_q8_1):
        with pytest.raises(ValueError, match=f"contiguous vector of {K} elements"):
            call(x, v)
    assert bool((mq.linear_f16cache(x, w, bias=v[:N]) == 1).all())


@pytest.mark.parametrize("past", [False, True])
@pytest.mark.parametrize("fmt", [synth.Q4_K, synth.Q5_K, synth.Q6_K, synth.Q5_1])
def test_far_gated_blocks(fmt, past):
    """Gated block weights on 256 x 256 tiles, past 2 GiB, which one buffer range
    from the gate rows to the weight's end cannot cover, and the largest that it
    can: rows at the edges of tiles, of 32-row blocks and of both halves, the
    rest zero."""
    K, M = 16384, 300
    row = mq.row_bytes(fmt, K)
    N = ((1 << 31) - 16) // (2 * row)
    if past:
        N = N // 256 * 256 + 301
    announce("glu far blocks", fmt, N)
    assert (2 * N * row + 16 > 1 << 31) == past
    p = mq.gemm_plan(fmt, M, 2 * N, K)
    assert (p["bm"], p["bn"]) == (256, 256)
    at = [0, 1, 31, 32, 63, 64, 127, 128, 4095, N // 2, N - 128, N - 46, N - 45, N - 2, N - 1]
    few = synth.weights(fmt, synth.rng(50, fmt), 2 * len(at), K)
    wb = oracle.dequant_ref(fmt, few, 2 * len(at), K)
    where = torch.tensor(at + [N + n for n in at], device=dev())
    q = torch.zeros(2 * N, row, dtype=torch.uint8, device=dev())
    q[where] = to_dev_u8(few).view(len(where), row)
    x, xb = _x(M, K, "f16", 51)
    bias = np.zeros(2 * N, np.float32)
    b = _vec(2 * len(at), 52)
    bias[np.array(at + [N + n for n in at])] = b
    y, g, u, Sg, Su = layers.glu_ref(xb, wb, K, b, "silu")
    eg, eu = 1.13 * _dv(K, Sg) + _da(g, "silu"), _dv(K, Su)
    err = eg * np.abs(u) + np.abs(layers.act_ref(g, "silu")) * eu + eg * eu
    tol = _out(y, err + U * (np.abs(y) + err), "f32")
    got = mq.glu_fused(x, q.view(-1), fmt, N, K, bias=torch.from_numpy(bias).to(dev()),
                       out_dtype=torch.float32)
    assert _worst(got[:, at], y, tol, "f32") <= 1
    got[:, at] = 0
    assert not bool(got.any())
    del q, got
    torch.cuda.empty_cache()


def _far_views(M, cols, ld, dtype, count):
    """`count` matrices of cols columns side by side in rows `ld` elements apart,
    each followed by 8 columns of NaN."""
    buf = torch.empty(M * ld, dtype=dtype, device=dev()).view(M, ld)
    buf[:, :count * (cols + 8)] = float("nan")
    return buf, [buf[:, i * (cols + 8):i * (cols + 8) + cols] for i in range(count)]


@pytest.mark.parametrize("M,split", [(5, 0), (32, 0), (40, 1), (300, 1), (300, 3)])
def test_outputs_and_residuals_past_2_to_31_elements(M, split):
    """Rows of y and of the residual whose offsets pass 2^31 elements, as the last
    token's rows of long sequences are: few-row kernels, whole tiles and the
    reduce of a K split, in place and not."""
    N, K = 200, 512
    ld = ((1 << 31) // (M - 1) + 4096) | 1
    announce("far outputs", M, split, ld)
    w, _ = _weight(0, N, K, 60)
    x, _ = _x(M, K, "f16", 60)
    for dt in ("f32", "f16"):
        r = torch.from_numpy(_vec((M, N), 61)).to(dev()).to(T[dt])
        want = mq.linear_f16cache(x, w, K, act="gelu", residual=r, split_k=split, out_dtype=T[dt])
        gated = mq.glu_f16cache(x, w, K, split_k=split, out_dtype=T[dt])
        buf, (rv, yv, gv) = _far_views(M, N, ld, T[dt], 3)
        assert (M - 1) * buf.stride(0) >= 1 << 31
        rv.copy_(r)
        kw = dict(act="gelu", residual=rv, split_k=split)
        mq.linear_f16cache(x, w, K, out=yv, **kw)
        mq.glu_f16cache(x, w, K, split_k=split, out=gv[:, :N // 2])
        assert torch.equal(yv, want) and torch.equal(gv[:, :N // 2], gated)
        assert torch.equal(rv, r)
        mq.linear_f16cache(x, w, K, out=rv, **kw)
        assert torch.equal(rv, want)
        assert int(torch.isnan(buf[:, :3 * (N + 8)]).sum()) == M * (24 + N // 2)
        del buf, rv, yv, gv, kw
        torch.cuda.empty_cache()


@pytest.mark.parametrize("K", [200, 3584, 33000])
def test_norm_rows_past_2_to_31_elements(K):
    """The same of the norm's rows: x, the stream in and out, and y."""
    M = 4
    ld = ((1 << 31) // (M - 1) + 4096) | 1
    announce("far norm rows", K)
    w = torch.from_numpy(1 + _vec(K, 62, 0.2)).to(dev())
    for dt in ("f32", "f16"):
        x = torch.from_numpy(_vec((M, K), 63)).to(dev()).to(T[dt])
        r = torch.from_numpy(_vec((M, K), 64)).to(dev()).to(T[dt])
        y, h = mq.add_rms_norm(x, w, residual=r, out_dtype=T[dt])
        buf, (xv, rv, hv, yv) = _far_views(M, K, ld, T[dt], 4)
        xv.copy_(x)
        rv.copy_(r)
        mq.add_rms_norm(xv, w, residual=rv, out=yv, residual_out=hv)
        assert torch.equal(yv, y) and torch.equal(hv, h) and torch.equal(rv, r)
        mq.add_rms_norm(xv, w, residual=rv, out=yv, residual_out=rv)
        assert torch.equal(yv, y) and torch.equal(rv, h) and torch.equal(xv, x)
        assert int(torch.isnan(buf[:, :4 * (K + 8)]).sum()) == M * 32
        if K % 32 == 0:
            xq, ds, _ = mq.add_rms_norm_q8_1(xv, w, residual=hv, residual_out=rv)
            eq, eds, eh = mq.add_rms_norm_q8_1(x, w, residual=h)
            assert torch.equal(xq, eq) and torch.equal(ds, eds) and torch.equal(rv, eh)
        del buf, xv, rv, hv, yv
        torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", [synth.Q4_K, synth.Q5_K, synth.Q6_K])
def test_few_rows_see_extreme_super_block_scales(fmt):
    """Super-block scales (and Q4_K's and Q5_K's offsets) from the smallest
    subnormal to the largest whose values stay finite, of both signs, and zero,
    in every pairing: the few-row kernels and the tile kernel expand the decode's
    values."""
    N, K = 182, 512
    announce("one-hot, extreme super-block scales", fmt)
    q = synth.weights(fmt, synth.rng(53, fmt), N, K).copy()
    blocks = q.reshape(-1, mq.block_bytes(fmt))
    scales = np.array([0x0001, 0x0003, 0x00FF, 0x03FF, 0x0400, 0x0401, 0x07FF, 0x1234, 0x3555,
                       0x3C01, 0x47FE, 0x4BFF if fmt == synth.Q6_K else 0x4FFF, 0x8001, 0x83FF,
                       0x8401, 0xB7FD, 0xC7FE, 0x0000, 0x8000], np.uint16)
    n = np.arange(len(blocks))
    d = scales[n % len(scales)].view(np.uint8).reshape(-1, 2)
    if fmt == synth.Q6_K:
        blocks[:, 208:] = d
        blocks[::3, 192:208] = np.array([0x80, 0x7F] * 8, np.uint8)      # -128 and 127
    else:
        blocks[:, :2] = d
        blocks[:, 2:4] = scales[n // len(scales) % len(scales)].view(np.uint8).reshape(-1, 2)
        assert len(blocks) >= len(scales) ** 2
        blocks[::3, 4:16] = 0xFF                                          # 63 and 63
    want = oracle.dequant_ref(fmt, q, N, K).view(np.float16).astype(np.float32)
    assert np.isfinite(want).all() and np.abs(want).max() > 3e4
    w = to_dev_u8(q)
    eye = torch.eye(K, dtype=torch.float16, device=dev())
    for rows in (4, 8, 16, 32, 64):
        got = torch.cat([mq.linear_fused(eye[k:k + rows], w, fmt, N, K)
                         for k in range(0, K, rows)])
        assert np.array_equal(got.t().cpu().numpy(), want), rows
    got = torch.cat([mq.linear_fused(eye[k:k + 4].float(), w, fmt, N, K) for k in range(0, K, 4)])
    assert np.array_equal(got.t().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", [0] + FMTS)
@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_few_rows_keep_special_values_apart(fmt, xt):
    """NaN and infinities of one activation row stay in that row of y, and those
    of one weight row in that column, in every few-row kernel; a part unit's
    cleared elements bring none in."""
    N, K = 50, 512 if fmt in (synth.Q4_K, synth.Q5_K, synth.Q6_K) else 288
    announce("special values, few rows", fmt, xt)
    w, _ = _weight(fmt, 2 * N, K, 70)
    bad_w = w.clone()
    if fmt == 0:
        bad_w[7, :K] = float("inf")
    else:
        row, at = mq.row_bytes(fmt, K), 208 if fmt == synth.Q6_K else 0
        for i in range(0, row, mq.block_bytes(fmt)):
            bad_w.view(2 * N, row)[7, i + at:i + at + 2] = torch.tensor([0, 0x7C], device=dev())

    def run(x, w, glu):
        if fmt == 0:
            return mq.glu_f16cache(x, w, K, act="relu", out_dtype=torch.float32) if glu else \
                mq.linear_f16cache(x, w, K, act="relu")
        f = mq.glu_fused if glu else mq.linear_fused
        return f(x, w, fmt, N if glu else 2 * N, K, act="relu", out_dtype=torch.float32)

    for M in (3, 4, 7, 11, 16, 19, 32):
        x, _ = _x(M, K, xt, M)
        bad = x.clone()
        bad[1, 7], bad[2, K - 1] = float("nan"), float("inf")
        keep = [i for i in range(M) if i not in (1, 2)]
        for glu in (False, True):
            want = run(x, w, glu)
            assert bool(torch.isfinite(want).all())
            y = run(bad, w, glu)
            assert torch.equal(y[keep], want[keep]), M
            assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[2]).all())
            y = run(x, bad_w, glu)
            cols = [c for c in range(want.shape[1]) if c != 7]
            assert torch.equal(y[:, cols], want[:, cols]), M
            if fmt == 0:                             # infinities of both signs
                assert bool(torch.isnan(y[:, 7]).all())


def test_splits_beyond_int_are_refused():
    """With a workspace of the caller's, which no size query precedes."""
    K, N, split = 512, 64, (1 << 32) + 2
    announce("splits beyond int")
    x = torch.zeros(40, K, dtype=torch.float16, device=dev())
    w = torch.zeros(N, K, dtype=torch.float16, device=dev())
    q = torch.zeros(N * mq.row_bytes("q8_0", K), dtype=torch.uint8, device=dev())
    ws = torch.empty(1 << 22, device=dev())
    xq, ds = mq.quantize_q8_1(x.float())
    for call in (lambda: mq.gemm_f16cache(x, w, K, split_k=split, ws=ws),
                 lambda: mq.gemm_fused(x, q, "q8_0", N, K, split_k=split, ws=ws),
                 lambda: mq.gemm_mmq(xq, ds, q, "q8_0", N, K, split_k=split, ws=ws),
                 lambda: mq.linear_f16cache(x, w, K, split_k=split, ws=ws),
                 lambda: mq.glu_fused(x, q, "q8_0", N // 2, K, split_k=split, ws=ws)):
        with pytest.raises(mq.MQError) as e:
            call()
        assert e.value.code == _lib.MQ_ERR_SPLIT
