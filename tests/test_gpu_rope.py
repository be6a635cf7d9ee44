"""Rotary positions on the GPU against the f64 oracle.

Tolerance.  u = 2^-24.  Cosine and sine are rounded once to f32 (their f64 sums are off
by about 1e-13), each of the two products and their sum once more: at most
(|x0| + |x1|)·|mscale|·(u + u) + u·|y|, where |y| <= (|x0| + |x1|)·|mscale|: 3u of that
(1.01 for the products of small terms).  An f16 output adds its rounding, 2^-11 of the
value (2^-25 absolute below the smallest normal).  Elements behind the rotated ones are
copied: rounded alone."""

import numpy as np
import pytest

from gpu_common import announce, dev, needs_gpu, to_host
from oracle import attention as oa

pytestmark = [pytest.mark.gpu, needs_gpu]

import torch  # noqa: E402

import quantized_weight_prefill_q4_amd as mq  # noqa: E402

U = 2.0 ** -24
T = {"f32": torch.float32, "f16": torch.float16}


def _check(M, H, D, n_rot, layout, xt, yt, pad=0, lead=0, mscale=1.0, pos=None, in_place=False):
    announce("rope", M, H, D, n_rot, layout, xt, yt, "pad", pad, "lead", lead, in_place)
    g = torch.Generator(device=dev()).manual_seed(M * 31 + D)
    W = H * D
    buf = torch.randn(M * (W + pad) + lead, generator=g, device=dev()).to(T[xt])
    x = buf[lead:].view(M, W + pad)[:, :W]
    if pos is None:
        pos = torch.randint(-5, 200000, (M,), generator=g, device=dev(), dtype=torch.int32)
    f = mq.rope_freqs(n_rot, device=dev())
    xs = to_host(x).astype(np.float64).reshape(M, H, D)
    m32 = float(np.float32(mscale))
    ref = oa.rotate_ref(xs, to_host(pos), to_host(f), layout, m32)
    n = n_rot // 2
    part = np.abs(xs)
    tol = np.zeros_like(ref)
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else \
        (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    both = (part[..., a] + part[..., b]) * abs(m32) * 3 * U * 1.01
    tol[..., a], tol[..., b] = both, both
    if yt == "f16":
        tol += 2.0 ** -11 * (np.abs(ref) + tol) + 2.0 ** -25
    guard = torch.full((M * (W + pad) + lead,), 77, device=dev()).to(T[yt])
    out = x if in_place else guard[lead:].view(M, W + pad)[:, :W]
    behind = buf.clone()
    y = mq.rope(x, pos, f, D, layout=layout, mscale=mscale, out=out)
    assert y is out
    got = to_host(y).astype(np.float64).reshape(M, H, D)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], np.abs(got - ref).max())
    if in_place:                       # the columns between the rows are as they were
        mask = torch.ones_like(behind, dtype=torch.bool)
        mask[lead:].view(M, W + pad)[:, :W] = False
        assert torch.equal(buf[mask], behind[mask])
    else:
        assert torch.equal(buf, behind)
        assert int((guard == 77).sum()) >= M * pad + lead
        fresh = mq.rope(x, pos, f, D, layout=layout, mscale=mscale, out_dtype=T[yt])
        assert torch.equal(fresh, y)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("xt,yt", [("f16", "f16"), ("f32", "f32"), ("f32", "f16"), ("f16", "f32")])
def test_types_and_layouts(layout, xt, yt):
    for H, D, n in ((1, 128, 128), (3, 64, 32), (2, 96, 96), (5, 80, 34), (2, 7, 6), (1, 2, 2),
                    (2, 33, 18)):
        _check(5, H, D, n, layout, xt, yt, pad=3, lead=1)


@pytest.mark.parametrize("M", [1, 2, 255, 1023, 1024, 1027])
def test_row_counts(M):
    _check(M, 3, 128, 128, "half", "f16", "f16")
    _check(M, 2, 64, 16, "interleaved", "f32", "f32", pad=8)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_and_magnitude(layout):
    for xt in ("f16", "f32"):
        _check(9, 4, 128, 64, layout, xt, xt, pad=512, mscale=1.139, in_place=True)
        _check(1030, 2, 64, 64, layout, xt, xt, in_place=True)
        _check(1, 32, 128, 128, layout, xt, xt, pad=512, mscale=-0.5, in_place=True)
    _check(3, 1, 1024, 1024, layout, "f32", "f16")
    _check(1100, 1, 1024, 1024, layout, "f16", "f16")


def test_far_positions():
    ends = [0, 1, -1, 1000003, (1 << 31) - 1, -(1 << 31), (1 << 24) + 1, -99999]
    pos = torch.tensor(ends, dtype=torch.int32, device=dev())
    _check(len(ends), 2, 128, 128, "half", "f32", "f32", pos=pos)


def test_a_turn_and_back_and_special_values():
    announce("rope there and back")
    x = torch.randn(6, 256, device=dev())
    f = mq.rope_freqs(128, device=dev())
    p = torch.arange(6, device=dev(), dtype=torch.int32) * 70001
    y = mq.rope(mq.rope(x, p, f, 128), -p, f, 128)
    assert float((x - y).abs().max()) < 16 * U * float(x.abs().max())
    z = mq.rope(x, torch.zeros_like(p), f, 128)
    assert torch.equal(z, x)
    x[2, 5], x[3, 7] = float("inf"), float("nan")        # pairs with 5 + 64 and 7 + 64, head 0
    y = mq.rope(x, p, f, 128)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[2, [5, 69]] = want[3, [7, 71]] = True
    assert torch.equal(bad, want)


def test_streams_and_graphs():
    announce("rope on another stream, captured and replayed")
    x = torch.randn(33, 4096, device=dev()).half()
    f = mq.rope_freqs(128, device=dev())
    p = torch.arange(33, device=dev(), dtype=torch.int32)
    y = mq.rope(x, p, f, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2 = mq.rope(x, p, f, 128)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2)
    out, g = torch.empty_like(y), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.rope(x, p, f, 128, out=out)
    for rep in range(3):
        out.fill_(1)
        p.add_(1000)
        want = mq.rope(x, p, f, 128)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep
    del g


def test_refusals():
    announce("rope refusals")
    x, f = torch.randn(4, 128, device=dev()), mq.rope_freqs(64, device=dev())
    p = torch.zeros(4, dtype=torch.int32, device=dev())
    for kw, text in ((dict(x=x.cpu()), "GPU tensor"), (dict(x=x.double()), "float32 or float16"),
                     (dict(x=x[0]), "2-D"), (dict(x=x.t()), "unit column stride"),
                     (dict(positions=p.long()), "positions must be Int"),
                     (dict(positions=p[:3]), "positions must be a contiguous vector"),
                     (dict(positions=p.cpu()), "same GPU"), (dict(freqs=f.float()), "freqs must be Double"),
                     (dict(freqs=f.cpu()), "same GPU"), (dict(freqs=f[::2]), "contiguous vector"),
                     (dict(head_dim=60), "multiple of head_dim"), (dict(head_dim=0), "head_dim"),
                     (dict(out=x[:3]), "out must be at least"), (dict(out=x.int()), "float32 or"),
                     (dict(out=x.cpu()), "same GPU"), (dict(layout=1), "unknown layout")):
        a = {**dict(x=x, positions=p, freqs=f, head_dim=64), **kw}
        with pytest.raises(ValueError, match=text):
            mq.rope(**a)
    for kw, code in ((dict(x=x[:0], positions=p[:0]), mq._lib.MQ_ERR_SHAPE),
                     (dict(freqs=f[:0]), None), (dict(head_dim=32), mq._lib.MQ_ERR_SHAPE),
                     (dict(mscale=float("nan")), mq._lib.MQ_ERR_EPS),
                     (dict(x=x[:1].expand(4, 128)), mq._lib.MQ_ERR_LD),
                     (dict(out=x[:, :].half().new_empty(0)), None)):
        a = {**dict(x=x, positions=p, freqs=f, head_dim=64), **kw}
        with pytest.raises((mq.MQError, ValueError)) as e:
            mq.rope(**a)
        if code is not None:
            assert e.value.code == code
