"""The residual RMS norm on the GPU against the f64 oracle.

Tolerances.  u = 2^-24.  The sum of squares adds at most 8·C elements per
thread in a chain (C <= 4 chunks; K / 1024 of them beyond 32768 elements),
then 6 shuffle and at most 15 cross-wave additions: its relative error is at
most (chain + 21 + 1)·u, which the square root halves; the mean, the sum with
eps, the root, the reciprocal and the two products add at most 6·u.  An f16
output adds its rounding, 2^-11 of the value (2^-25 absolute below the
smallest normal).  h is exact: one f32 addition, rounded to the stream's type.
"""

import numpy as np
import pytest

from gpu_common import announce, dev, needs_gpu, to_host
from oracle import layers

pytestmark = [pytest.mark.gpu, needs_gpu]

import torch  # noqa: E402

import quantized_weight_prefill_q4_amd as mq  # noqa: E402

U = 2.0 ** -24
T = {"f32": torch.float32, "f16": torch.float16}


def _tol(y, K, out):
    chain = 32 if K <= 32768 else 8 * ((K // 8 + 1023) // 1024 + 1)
    t = ((chain + 22) / 2 + 6) * U * np.abs(y)
    if out == "f16":
        t = t * (1 + 2.0 ** -11) + 2.0 ** -11 * np.abs(y) + 2.0 ** -25
    return t + 1e-44


def _strided(t, pad, lead):
    """The same matrix inside a wider buffer of NaN, `lead` elements in."""
    M, K = t.shape
    buf = torch.full((M * (K + pad) + lead,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[lead:].view(M, K + pad)[:, :K]
    v.copy_(t)
    return buf, v


def _inputs(M, K, xt, rt, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=dev()).to(T[xt])
    r = None if rt is None else (3 * torch.randn(M, K, generator=g, device=dev())).to(T[rt])
    w = 1 + 0.3 * torch.randn(K, generator=g, device=dev())
    return x, r, w


def _check(M, K, xt, rt, yt, pad, lead, eps=1e-6):
    announce("add_rms_norm", M, K, xt, rt, yt, "pad", pad, "lead", lead)
    x, r, w = _inputs(M, K, xt, rt, M * 7 + K)
    ref_y, ref_h = layers.rms_norm_ref(to_host(x), to_host(w), eps,
                                       None if r is None else to_host(r))
    _, xv = _strided(x, pad, lead)
    rv = None if r is None else _strided(r, pad, lead)[1]
    ybuf, yv = _strided(torch.zeros(M, K, dtype=T[yt], device=dev()), pad, lead)
    hbuf = hv = None
    if r is not None:
        hbuf, hv = _strided(torch.zeros_like(r), pad, lead)
    y, h = mq.add_rms_norm(xv, w, residual=rv, eps=eps, out=yv, residual_out=hv)
    assert y is yv and h is hv
    got = to_host(yv).astype(np.float64)
    worst = np.max(np.abs(got - ref_y) / _tol(ref_y, K, yt))
    assert worst <= 1, f"y {worst:.3g} times its tolerance"
    # nothing but the K columns of each row was written
    assert int(torch.isnan(ybuf).sum()) == lead + M * pad
    if r is not None:
        assert np.array_equal(to_host(hv).astype(np.float64), ref_h)
        assert int(torch.isnan(hbuf).sum()) == lead + M * pad
    y2, h2 = mq.add_rms_norm(x, w, residual=r, eps=eps, out_dtype=T[yt])
    assert torch.equal(y2, yv) and (r is None or torch.equal(h2, hv))


@pytest.mark.parametrize("K", [1, 2, 7, 8, 9, 31, 64, 100, 511, 512, 513, 1001, 2048, 2049, 3584,
                               4096, 4097, 8192, 8200, 16384, 16385, 32768, 32769, 40003])
def test_widths(K):
    for M in (1, 5):
        _check(M, K, "f32", "f32", "f16", 0, 0)
        _check(M, K, "f16", "f16", "f32", 3, 1)


@pytest.mark.parametrize("xt", ["f32", "f16"])
@pytest.mark.parametrize("rt", [None, "f32", "f16"])
@pytest.mark.parametrize("yt", ["f32", "f16"])
def test_types(xt, rt, yt):
    for K, pad, lead in ((3584, 0, 0), (1001, 7, 0), (1000, 1, 3), (37, 5, 1)):
        _check(9, K, xt, rt, yt, pad, lead)


@pytest.mark.parametrize("M", [1, 3, 4, 17, 255, 1030, 4099])
def test_row_counts(M):
    _check(M, 1001, "f16", "f16", "f16", 7, 0)
    _check(M, 3584, "f32", "f32", "f16", 0, 0)
    _check(M, 96, "f32", None, "f32", 0, 0)
    _check(M, 200, "f16", "f32", "f16", 1, 1)
    _check(M, 2300, "f16", "f32", "f32", 0, 0)


@pytest.mark.parametrize("M,K", [(1, 32), (1, 3584), (3, 96), (7, 4096), (300, 3584), (2, 16384),
                                 (2, 32800), (1029, 512)])
@pytest.mark.parametrize("rt", [None, "f32", "f16"])
def test_q8_1_is_the_quantized_norm(M, K, rt):
    """The codes and factors are quantize_q8_1's of the f32 norm, bit for bit."""
    announce("add_rms_norm_q8_1", M, K, rt)
    x, r, w = _inputs(M, K, "f16" if K == 96 else "f32", rt, M + K)
    xv = _strided(x, 3, 1)[1]
    y, h = mq.add_rms_norm(x, w, residual=r, out_dtype=torch.float32)
    xq, ds, hq = mq.add_rms_norm_q8_1(xv, w, residual=r)
    eq, eds = mq.quantize_q8_1(y)
    assert torch.equal(xq[:, :K], eq[:, :K]) and torch.equal(ds, eds)
    assert h is None and hq is None or torch.equal(h, hq)
    wide = torch.full((M, K + 16), 77, dtype=torch.int8, device=dev())
    mq.add_rms_norm_q8_1(x, w, residual=r, xq=wide)
    assert torch.equal(wide[:, :K], eq[:, :K]) and bool((wide[:, K:] == 77).all())


def test_feeds_the_int8_product():
    """The norm's blocks go straight into the int8 product."""
    import synth
    M, N, K = 5, 64, 512
    announce("norm -> gemm_mmq")
    q = torch.from_numpy(synth.weights(synth.Q4_K, synth.rng(7), N, K)).to(dev()).reshape(-1)
    x, r, w = _inputs(M, K, "f32", "f32", 3)
    xq, ds, h = mq.add_rms_norm_q8_1(x, w, residual=r)
    y, _ = mq.add_rms_norm(x, w, residual=r, out_dtype=torch.float32)
    eq, eds = mq.quantize_q8_1(y)
    assert torch.equal(mq.gemm_mmq(xq, ds, q, "q4_k", N, K), mq.gemm_mmq(eq, eds, q, "q4_k", N, K))


@pytest.mark.parametrize("K", [3584, 1001, 40003])
def test_in_place(K):
    announce("add_rms_norm in place", K)
    x, r, w = _inputs(6, K, "f32", "f32", 11)
    y, h = mq.add_rms_norm(x, w, residual=r, out_dtype=torch.float32)
    for place in ("stream", "x and stream", "swapped"):
        x2, r2 = x.clone(), r.clone()
        if place == "stream":
            y2, h2 = mq.add_rms_norm(x2, w, residual=r2, out_dtype=torch.float32, residual_out=r2)
        elif place == "x and stream":
            y2, h2 = mq.add_rms_norm(x2, w, residual=r2, out=x2, residual_out=r2)
        else:
            y2, h2 = mq.add_rms_norm(x2, w, residual=r2, out=r2, residual_out=x2)
        assert torch.equal(y, y2) and torch.equal(h, h2), place
    both = torch.empty(6, 2 * K, device=dev())        # outputs side by side in one buffer
    y2, h2 = mq.add_rms_norm(x, w, residual=r, out=both[:, K:], residual_out=both[:, :K])
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_rows_do_not_touch_each_other():
    """A row of zeros gives zeros, rows with infinities or NaN stay alone."""
    announce("add_rms_norm special rows")
    K = 520
    x, r, w = _inputs(6, K, "f32", "f32", 12)
    clean, _ = mq.add_rms_norm(x, w, residual=r)
    x[1], r[1] = 0, 0
    x[2, 3] = float("inf")
    x[3, 519] = float("nan")
    x[4] *= 1e-30                                    # squares far below f32's range
    r[4] = 0
    y, h = mq.add_rms_norm(x, w, residual=r)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[5], clean[5])
    assert bool((y[1] == 0).all()) and bool((h[1] == 0).all())
    # inf: mean inf, 1/sqrt = 0: zeros but inf * 0 = NaN at the place itself
    assert bool(torch.isnan(y[2, 3])) and int(torch.isnan(y[2]).sum()) == 1
    assert bool((y[2].nan_to_num(0) == 0).all())
    assert bool(torch.isnan(y[3]).all())
    ref, _ = layers.rms_norm_ref(to_host(x[4:5]), to_host(w), 1e-6, to_host(r[4:5]))
    assert np.all(np.abs(to_host(y[4:5]) - ref) <= _tol(ref, K, "f16"))
    y0, _ = mq.add_rms_norm(x[1:2], w, eps=0.0)      # 0 / 0
    assert bool(torch.isnan(y0).all())


def test_streams_and_graphs():
    announce("add_rms_norm on another stream, captured and replayed")
    x, r, w = _inputs(33, 3584, "f32", "f32", 13)
    y, h = mq.add_rms_norm(x, w, residual=r)
    xq, ds, _ = mq.add_rms_norm_q8_1(x, w, residual=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, h2 = mq.add_rms_norm(x, w, residual=r)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    outs = [torch.empty_like(y), torch.empty_like(h), torch.empty_like(xq), torch.empty_like(ds)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.add_rms_norm(x, w, residual=r, out=outs[0], residual_out=outs[1])
        mq.add_rms_norm_q8_1(x, w, residual=r, xq=outs[2], ds=outs[3], residual_out=outs[1])
    for rep in range(3):
        for t in outs:
            t.fill_(1)
        x.mul_(0.5)
        r.mul_(0.5)
        want = [*mq.add_rms_norm(x, w, residual=r), *mq.add_rms_norm_q8_1(x, w, residual=r)[:2]]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), f"replay {rep}"
    del g


def test_binding_refuses():
    announce("add_rms_norm refusals")
    x, r, w = _inputs(4, 64, "f32", "f32", 14)
    for kw, text in ((dict(x=x.cpu()), "GPU tensor"), (dict(x=x.double()), "float32 or float16"),
                     (dict(x=x[0]), "2-D"), (dict(x=x.t()), "unit column stride"),
                     (dict(weight=w[:-1]), "contiguous vector"), (dict(weight=w.half()), "float32"),
                     (dict(weight=w.cpu()), "same GPU"),
                     (dict(residual=r[:3]), "residual must be at least"),
                     (dict(residual=r[:, :63]), "residual must be at least"),
                     (dict(residual=r.cpu()), "same GPU"), (dict(residual=r.int()), "float32 or"),
                     (dict(residual=None, residual_out=r), "needs a residual"),
                     (dict(residual_out=r.half()), "residual_out must be"),
                     (dict(out_dtype=torch.bfloat16), "out_dtype"),
                     (dict(out=torch.empty(4, 63, device=dev())), "out must be at least"),
                     (dict(out=torch.empty(4, 64, device=dev(), dtype=torch.int32)), "float32 or")):
        a = {**dict(x=x, weight=w, residual=r), **kw}
        with pytest.raises(ValueError, match=text):
            mq.add_rms_norm(**a)
    for kw, code in ((dict(eps=-1.0), mq._lib.MQ_ERR_EPS), (dict(out=r), None),
                     (dict(residual=r[:1].expand(4, 64)), mq._lib.MQ_ERR_LD),
                     (dict(residual_out=x, out=x), mq._lib.MQ_ERR_OVERLAP),
                     (dict(x=x[:0], residual=r[:0]), mq._lib.MQ_ERR_SHAPE)):
        a = {**dict(x=x, weight=w, residual=r.clone()), **kw}
        if code is None:
            mq.add_rms_norm(**a)
            continue
        with pytest.raises(mq.MQError) as e:
            mq.add_rms_norm(**a)
        assert e.value.code == code
    with pytest.raises(ValueError, match="xq must be torch.int8"):
        mq.add_rms_norm_q8_1(x, w, xq=torch.empty(4, 64, device=dev()))
    with pytest.raises(ValueError, match="ds must be"):
        mq.add_rms_norm_q8_1(x, w, ds=torch.empty(15, device=dev()))
    with pytest.raises(mq.MQError):
        mq.add_rms_norm_q8_1(x[:, :48], w)
