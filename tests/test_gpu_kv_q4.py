"""The 4-bit key/value cache's store and load on the GPU.

The store's codes and scales are compared with the oracle's bit for bit, read from the
cache's bytes at their documented places: the blocks are f32 steps that both sides take
alike, and so is the rotation (f64 angles, cosine and sine rounded once to f32, each
operation rounded once).  The load is exact in f32 and rounds once to f16."""

import numpy as np
import pytest

from gpu_common import announce, dev, needs_gpu, to_host
from oracle import attention as oa

pytestmark = [pytest.mark.gpu, needs_gpu]

import torch  # noqa: E402

import quantized_weight_prefill_q4_amd as mq  # noqa: E402

T = {"f32": torch.float32, "f16": torch.float16}
I32 = torch.int32


def ints(v):
    return torch.tensor(v, dtype=I32, device=dev())


class Batch:
    """Sequences over a cache whose pages are shuffled; every byte starts as 0xFF
    (codes 15, scales NaN)."""

    def __init__(self, D, Hkv, page, rows, lens, seed=0, ragged=True, stride=0):
        rng = np.random.default_rng(seed)
        self.D, self.Hkv, self.page, self.rows, self.lens = D, Hkv, page, rows, lens
        need = [-(-n // page) for n in lens]
        self.width = max(need) + 1
        pages = sum(need) + 2
        order = rng.permutation(pages)[:sum(need)]
        table, at = np.full((len(lens), self.width), -1, np.int32), 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k
        self.table_np, self.table = table, torch.from_numpy(table).to(dev())
        per = mq.kv_page_bytes(Hkv, page, D) + stride
        self.bytes = torch.full((pages, per), 255, dtype=torch.uint8, device=dev())
        tiles = page // 32
        self.cache = self.bytes.as_strided((pages, Hkv, tiles, 36 * D),
                                           (per, tiles * 36 * D, 36 * D, 1))
        self.lens_t = ints(lens)
        self.cu_np = np.concatenate(([0], np.cumsum(rows)))
        self.cu = ints(self.cu_np.tolist()) if ragged else None
        self.M = sum(rows)

    def positions(self):
        return np.concatenate([np.arange(n - r, n) for r, n in zip(self.rows, self.lens)])

    def tokens(self):
        """(key codes, key d, value codes, value d) of each sequence's tokens."""
        kc, kd, vc, vd = oa.cache_tokens(to_host(self.cache), self.D)
        out = []
        for b, n in enumerate(self.lens):
            p = self.table_np[b, np.arange(n) // self.page]
            o = np.arange(n) % self.page
            out.append([a[p, :, o] for a in (kc, kd, vc, vd)])
        return out


def rows_of(M, W, dtype, seed, pad=0, lead=0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    buf = torch.randn(M * (W + pad) + lead, generator=g, device=dev()).to(dtype)
    return buf[lead:].view(M, W + pad)[:, :W]


def _check(D, Hkv, page, rows, lens, xt, ragged=True, freqs=None, layout="half", pos=None, H=0,
           pad=0, lead=0, mscale=1.0, stride=0):
    announce("kv_store_q4", D, Hkv, page, rows, lens, xt, ragged, layout, "q heads", H)
    s = Batch(D, Hkv, page, rows, lens, D + page, ragged, stride)
    k, v = (rows_of(s.M, Hkv * D, T[xt], i, pad, lead) for i in (1, 2))
    q = rows_of(s.M, H * D, T[xt], 3, pad, lead) if H else None
    before = to_host(s.bytes).copy()
    qr = mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t, cu_rows=s.cu, freqs=freqs, layout=layout,
                        positions=pos, q=q, mscale=mscale)
    at = s.positions() if pos is None else to_host(pos)
    kf = to_host(k).astype(np.float32).reshape(s.M, Hkv, D)
    vf = to_host(v).astype(np.float32).reshape(s.M, Hkv, D)
    if freqs is not None:
        kf = oa.rotate_f32(kf, at, to_host(freqs), layout, mscale)
    want = oa.quantize_q4(kf) + oa.quantize_q4(vf)
    got = s.tokens()
    for b, (r, n) in enumerate(zip(rows, lens)):
        sl = slice(s.cu_np[b], s.cu_np[b] + r)
        for i, name in enumerate(("key codes", "key d", "value codes", "value d")):
            g = got[b][i]
            assert np.array_equal(g[n - r:n], want[i][sl]), (b, name)
            # what was there before is untouched
            rest = g[:n - r]
            assert (rest == 15).all() if i % 2 == 0 else np.isnan(rest).all(), (b, name)
    # and no other byte of the cache: count the tokens written
    new = Batch(D, Hkv, page, rows, lens, D + page, ragged, stride)
    changed = int((to_host(s.bytes) != before).sum())
    assert changed <= s.M * Hkv * 2 * (D + D // 16)
    assert torch.equal(s.bytes[:, new.bytes.shape[1] - stride:],
                       new.bytes[:, new.bytes.shape[1] - stride:])
    if H:
        assert qr.dtype == torch.float16
        qf = to_host(q).astype(np.float32).reshape(s.M, H, D)
        if freqs is not None:
            qf = oa.rotate_f32(qf, at, to_host(freqs), layout, mscale)
        assert np.array_equal(to_host(qr).reshape(s.M, H, D), qf.astype(np.float16))
    else:
        assert qr is None
    for yt in ("f32", "f16"):
        lk, lv = mq.kv_load_q4(s.cache, s.table, s.lens_t, s.M, cu_rows=s.cu, out_dtype=T[yt])
        for t, (c, d) in ((lk, want[:2]), (lv, want[2:])):
            ref = oa.values(c, d).astype(np.float32 if yt == "f32" else np.float16)
            assert np.array_equal(to_host(t).reshape(ref.shape), ref, equal_nan=True), yt
    return s, k, v


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("xt", ["f16", "f32"])
def test_head_sizes(D, xt):
    _check(D, 2, 32, [1, 7, 8, 40], [1, 20, 64, 73], xt)
    f = mq.rope_freqs(D, device=dev())
    _check(D, 3, 64, [9, 33], [9, 100], xt, freqs=f, H=6, pad=3, lead=1)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n_rot", [128, 64, 34, 2])
def test_rotations(layout, n_rot):
    f = mq.rope_freqs(n_rot, scale=2.0, device=dev())
    for xt in ("f16", "f32"):
        _check(128, 2, 32, [5, 1, 30], [40, 1000, 30], xt, freqs=f, layout=layout, H=5, mscale=1.07)


def test_one_row_each_and_equal_rows():
    f = mq.rope_freqs(128, device=dev())
    lens = [1, 2, 31, 32, 33, 65, 96, 97, 500, 8, 9, 7]
    _check(128, 4, 32, [1] * 12, lens, "f16", ragged=False, freqs=f, H=28)
    _check(128, 4, 32, [1] * 12, lens, "f32", ragged=True, freqs=f, H=28)
    _check(64, 1, 96, [13] * 4, [13, 14, 100, 97], "f16", ragged=False)
    _check(128, 8, 256, [700], [1500], "f16", ragged=False, freqs=f, H=8)


def test_prompts_whose_workgroups_take_several_heads():
    f = mq.rope_freqs(64, device=dev())
    _check(64, 5, 64, [2700], [2750], "f32", ragged=False, freqs=f, H=5)      # two heads each
    _check(64, 5, 64, [4000, 3001], [4000, 3100], "f16", freqs=f, H=5)        # four and one
    _check(128, 8, 128, [2100, 3100], [2111, 3100], "f32")


def test_many_sequences():
    rng = np.random.default_rng(4)
    rows = [int(r) for r in rng.integers(0, 4, 200)]
    _check(64, 2, 32, rows, [r + int(p) for r, p in zip(rows, rng.integers(0, 70, 200))], "f16")


def test_codes_of_all_magnitudes():
    """The quotient x/d is the correctly rounded one: blocks from 10^-9 to 10^4."""
    announce("kv_store_q4 magnitudes")
    s = Batch(128, 8, 64, [2048], [2048], 5, ragged=False)
    size = 10.0 ** (torch.rand(2048, 8 * 128 // 32, device=dev(), dtype=torch.float64) * 13 - 9)
    size = size.float().repeat_interleave(32, dim=1)
    k, v = (rows_of(2048, 8 * 128, torch.float32, i) * size for i in (1, 2))
    v = torch.where(torch.rand(v.shape, device=dev()) < 0.1, v * 1e-30, v)   # and tiny ones in them
    mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t)
    want = oa.quantize_q4(to_host(k).reshape(-1, 8, 128)) + oa.quantize_q4(to_host(v).reshape(-1, 8, 128))
    for g, w in zip(s.tokens()[0], want):
        assert np.array_equal(g, w, equal_nan=g.dtype.kind == "f")


def test_positions_of_their_own():
    f = mq.rope_freqs(96, device=dev())
    pos = ints([5, 900000, -3, 17, 2, 1])
    _check(96, 2, 32, [4, 2], [50, 2], "f32", freqs=f, pos=pos, H=2)


def test_empty_sequences_and_strided_pages():
    _check(128, 2, 32, [0, 3, 0, 0, 20, 0], [0, 3, 50, 0, 90, 32], "f16", stride=16)
    _check(64, 2, 64, [2, 0], [2, 9], "f32", stride=4096)


def test_token_by_token_is_the_prompt():
    """Appending one by one leaves the bytes that one call leaves: nibbles that share a
    dword with earlier tokens' included."""
    announce("kv_store_q4 token by token")
    f = mq.rope_freqs(128, device=dev())
    whole, k, v = _check(128, 2, 32, [45], [45], "f16", ragged=False, freqs=f)
    s = Batch(128, 2, 32, [45], [45], 160)
    at = 0
    for n in (1, 1, 1, 5, 8, 3, 1, 12, 1, 1, 11):
        mq.kv_store_q4(k[at:at + n], v[at:at + n], s.cache, s.table, ints([at + n]), freqs=f)
        at += n
    assert at == 45 and torch.equal(s.table, whole.table)
    assert torch.equal(s.bytes, whole.bytes)


def test_special_blocks():
    announce("kv_store_q4 special blocks")
    s = Batch(64, 1, 32, [8], [8], 3, False)
    k = rows_of(8, 64, torch.float32, 4).contiguous()
    v = rows_of(8, 64, torch.float32, 5).contiguous()
    k[0] = 0                                           # d = 0
    k[1, :32] = torch.tensor([1.0, -1.0] * 16)         # a tie: the first decides
    k[2, 3], k[2, 40] = float("nan"), float("inf")
    k[3] *= 1e-9                                       # d below f16
    k[4] *= 1e7                                        # d beyond f16
    v[5, 63] = float("-inf")
    v[6, :32] = torch.tensor([-2.0, 2.0] * 16)
    v[7] *= 3e-6                                       # subnormal d
    mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t)
    got = s.tokens()[0]
    want = oa.quantize_q4(to_host(k)[:, None]) + oa.quantize_q4(to_host(v)[:, None])
    for g, w in zip(got, want):
        assert np.array_equal(g, w, equal_nan=g.dtype != np.uint8)
    lk, lv = mq.kv_load_q4(s.cache, s.table, s.lens_t, 8)
    assert bool(torch.isnan(lk[2]).all()) and bool((lk[0] == 0).all())
    assert bool(torch.isnan(lv[5, 32:]).all()) and bool(torch.isfinite(lv[5, :32]).all())


def test_blocks_end_where_f16_does():
    """Elements up to 65519 are stored, a block with a larger one is NaN; for keys that is the
    element after its rotation, f16's own largest numbers included."""
    announce("kv_store_q4 blocks at the end of f16")
    tops = [60000.0, 65504.0, 65519.0, 65519.99609375, 65520.0, 65536.0, 1e5, 524000.0]
    s = Batch(64, 1, 32, [16], [16], 6, False)
    k = rows_of(16, 64, torch.float32, 7).contiguous() * 1000
    v = rows_of(16, 64, torch.float32, 8).contiguous() * 1000
    for i, top in enumerate(tops):
        for j, sign in enumerate((-1, 1)):
            k[i + 8 * j, 5], v[i + 8 * j, 40] = sign * top, -sign * top
    mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t)
    want = oa.quantize_q4(to_host(k)[:, None]) + oa.quantize_q4(to_host(v)[:, None])
    for g, w in zip(s.tokens()[0], want):
        assert np.array_equal(g, w, equal_nan=g.dtype != np.uint8)
    lk, lv = mq.kv_load_q4(s.cache, s.table, s.lens_t, 16)
    nan = torch.tensor([t >= 65520 for t in tops] * 2, device=dev())
    for t, block in ((lk, 0), (lv, 1)):
        t = t.view(16, 2, 32)
        assert torch.equal(torch.isnan(t[:, block]).all(1), nan)
        assert bool(torch.isfinite(t[:, block][~nan]).all()) and bool(torch.isfinite(t[:, 1 - block]).all())
    # f16 keys turned past f16's end: (a, a) by an eighth of a turn is (0, 1.41·a)
    f = torch.full((32,), np.pi / 4, dtype=torch.float64, device=dev())
    k = torch.zeros(2, 64, dtype=torch.float16, device=dev())
    k[:, [3, 35]] = 46000.0
    k[1, [3, 35]] = 47000.0
    one = ints([1, 1])
    mq.kv_store_q4(k, k, s.cache, s.table, ints([2]), freqs=f, positions=one)
    lk, lv = mq.kv_load_q4(s.cache, s.table, ints([2]), 2)
    assert float(lk[0, 35]) > 65000 and bool(torch.isfinite(lk[0]).all())
    assert bool(torch.isnan(lk[1, 32:]).all()) and bool(torch.isfinite(lv).all())


def test_in_place_queries_in_one_buffer():
    """q, k and v as columns of one activation, q rotated where it stands."""
    announce("kv_store_q4 in one buffer")
    D, H, Hkv = 128, 4, 2
    s = Batch(D, Hkv, 32, [3, 6], [3, 40], 5)
    x = rows_of(9, (H + 2 * Hkv) * D, torch.float16, 6)
    f = mq.rope_freqs(D, device=dev())
    q, k, v = x[:, :H * D], x[:, H * D:(H + Hkv) * D], x[:, (H + Hkv) * D:]
    want = mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t, cu_rows=s.cu, freqs=f, q=q)
    ref = s.bytes.clone()
    kv = x[:, H * D:].clone()
    got = mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t, cu_rows=s.cu, freqs=f, q=q, q_out=q)
    assert got is q and torch.equal(q, want) and torch.equal(s.bytes, ref)
    assert torch.equal(x[:, H * D:], kv)
    plain = mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t, cu_rows=s.cu, q=q,
                           q_dtype=torch.float32)
    assert torch.equal(plain, q.float())               # no rotation: a copy


def test_bad_pages_lens_and_rows_are_left_out():
    """Entries that name no page, positions past the table and before 0, rows before the
    first sequence and behind the last: nothing is stored there, the rest is."""
    announce("kv_store_q4 bad pages")
    D, page = 64, 32
    s = Batch(D, 1, page, [40, 40], [40, 40], 7)
    pages = s.cache.shape[0]
    k, v = rows_of(90, D, torch.float16, 8), rows_of(90, D, torch.float16, 9)
    q = rows_of(90, D, torch.float16, 10)
    f = mq.rope_freqs(D, device=dev())
    good = s.table.clone()
    for bad in (-1, pages, 1 << 30, -(1 << 31)):
        s.bytes.fill_(255)
        t = good.clone()
        t[0, 0] = bad                                  # tokens 0 .. 31 of sequence 0
        cu = ints([3, 43, 83])                         # rows 0 .. 2 and 83 .. 89: nobody's
        out = torch.full_like(q, 5)
        mq.kv_store_q4(k, v, s.cache, t, s.lens_t, cu_rows=cu, freqs=f, q=q, q_out=out)
        assert bool((out[:3] == 5).all()) and bool((out[83:] == 5).all())
        assert not bool((out[3:83] == 5).all(1).any())
        got = s.tokens()
        assert (got[0][2][:32] == 15).all() and np.isnan(got[0][1][:32]).all()
        wk = oa.quantize_q4(oa.rotate_f32(to_host(k)[35:43, None], np.arange(32, 40), to_host(f)))
        assert np.array_equal(got[0][0][32:40], wk[0])
        wv = oa.quantize_q4(to_host(v)[43:83, None])
        assert np.array_equal(got[1][2], wv[0])
        a, b = torch.full((90, D), 5.0, device=dev()), torch.full((90, D), 5.0, device=dev())
        mq.kv_load_q4(s.cache, t, s.lens_t, 90, cu_rows=cu, k_out=a, v_out=b)
        for x in (a, b):
            assert bool((x[:3] == 5).all()) and bool((x[83:] == 5).all())
            assert bool((x[3:35] == 0).all()) and not bool((x[35:83] == 5).any())
    # 40 rows of sequences of 10, 0 and fewer tokens: the last ones alone have a place
    s.bytes.fill_(255)
    out = torch.full_like(q, 5)
    mq.kv_store_q4(k[:80], v[:80], s.cache, good, ints([10, -3]), cu_rows=ints([0, 40, 80]), freqs=f,
                   q=q[:80], q_out=out[:80])
    assert bool((out[:30] == 5).all()) and bool((out[40:] == 5).all())
    got = s.tokens()
    assert np.array_equal(got[0][2][:10], oa.quantize_q4(to_host(v)[30:40, None])[0])
    assert (got[0][2][10:] == 15).all() and (got[1][2] == 15).all()
    # a table of two pages, a sequence of 80: positions 64 .. 79 have none
    s.bytes.fill_(255)
    t = good[:1, :2].contiguous()
    mq.kv_store_q4(k[:40], v[:40], s.cache, t, ints([80]))
    lk, _ = mq.kv_load_q4(s.cache, t, ints([80]), 40)
    want = oa.values(*oa.quantize_q4(to_host(k)[:24].astype(np.float32)))
    assert np.array_equal(to_host(lk)[:24], want.astype(np.float16))
    assert bool((lk[24:] == 0).all())


def test_far_pages():
    """A cache past 2^32 bytes."""
    D, Hkv, page = 128, 8, 256
    pages = (9 << 29) // mq.kv_page_bytes(Hkv, page, D) + 2
    announce("kv_store_q4 far pages", pages)
    cache = torch.empty((pages, Hkv, page // 32, 36 * D), dtype=torch.uint8, device=dev())
    k, v = rows_of(300, Hkv * D, torch.float16, 1), rows_of(300, Hkv * D, torch.float16, 2)
    outs = []
    for table in ([[0, 1]], [[pages - 1, pages - 2]]):
        mq.kv_store_q4(k, v, cache, ints(table), ints([300]))
        outs.append(mq.kv_load_q4(cache, ints(table), ints([300]), 300))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    want = oa.values(*oa.quantize_q4(to_host(v).astype(np.float32)))
    assert np.array_equal(to_host(outs[1][1]), want.astype(np.float16))


def test_sequences_without_rows_share_pages_with_others():
    """A slot without rows in the call whose length ends inside an octet (a finished request,
    a waiting fork) names a page that another sequence is stored into: the page is what that
    sequence leaves."""
    announce("kv_store_q4 idle slots over a page in use")
    for D, Hkv, n, idle in ((128, 8, 20, [13]), (64, 2, 32, [1, 7, 9, 15, 18, 25, 31, 33]),
                            (256, 4, 24, [5, 13, 21] * 40), (96, 3, 31, [30] * 70)):
        s = Batch(D, Hkv, 32, [n], [n], D, False)
        k, v = (rows_of(n, Hkv * D, torch.float16, i) for i in (1, 2))
        mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t)
        want = s.bytes.clone()
        B = len(idle)
        table = s.table.repeat(2 * B + 1, 1)
        lens = ints(idle + [n] + idle)
        cu = ints([0] * (B + 1) + [n] * (B + 1))
        lk, lv = mq.kv_load_q4(s.cache, s.table, s.lens_t, n)
        for _ in range(10):
            s.bytes.fill_(255)
            mq.kv_store_q4(k, v, s.cache, table, lens, cu_rows=cu)
            assert torch.equal(s.bytes, want), D
        a, b = mq.kv_load_q4(s.cache, table, lens, n, cu_rows=cu)
        assert torch.equal(a, lk) and torch.equal(b, lv)


def test_streams_and_graphs():
    announce("kv_store_q4 on another stream, captured and replayed")
    D, H, Hkv = 128, 4, 2
    s = Batch(D, Hkv, 32, [1, 1], [30, 31], 11, False)
    f = mq.rope_freqs(D, device=dev())
    k, v = rows_of(2, Hkv * D, torch.float16, 1), rows_of(2, Hkv * D, torch.float16, 2)
    q = rows_of(2, H * D, torch.float16, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t, freqs=f, q=q)
    torch.cuda.current_stream().wait_stream(side)
    bytes1 = s.bytes.clone()
    s.bytes.fill_(255)
    assert torch.equal(a, mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t, freqs=f, q=q))
    assert torch.equal(s.bytes, bytes1)
    out, g = torch.empty_like(q), torch.cuda.CUDAGraph()
    lk, lv = torch.empty_like(k), torch.empty_like(v)
    with torch.cuda.graph(g):
        mq.kv_store_q4(k, v, s.cache, s.table, s.lens_t, freqs=f, q=q, q_out=out)
        mq.kv_load_q4(s.cache, s.table, s.lens_t, 2, k_out=lk, v_out=lv)
    other = Batch(D, Hkv, 32, [1, 1], [30, 31], 11, False)
    other.bytes.copy_(bytes1)
    for rep in range(3):                               # a step further each time, onto a new page
        s.lens_t.add_(1)
        k.mul_(0.5)
        want = mq.kv_store_q4(k, v, other.cache, s.table, s.lens_t, freqs=f, q=q)
        wk, wv = mq.kv_load_q4(other.cache, s.table, s.lens_t, 2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(s.bytes, other.bytes), rep
        assert torch.equal(lk, wk) and torch.equal(lv, wv), rep
    del g


def test_refusals():
    announce("kv_store_q4 refusals")
    D, Hkv = 64, 2
    s = Batch(D, Hkv, 32, [2, 2], [2, 40], 12, False)
    k, v, q = (rows_of(4, n * D, torch.float16, i) for i, n in ((1, 2), (2, 2), (3, 4)))
    f = mq.rope_freqs(D, device=dev())
    base = dict(k=k, v=v, cache=s.cache, table=s.table, lens=s.lens_t, cu_rows=None, freqs=f, q=q)
    for kw, text in ((dict(k=k.cpu()), "GPU tensor"), (dict(v=v.cpu()), "same GPU"),
                     (dict(v=v.float()), "v must be Half"), (dict(k=k.double()), "float32 or float16"),
                     (dict(k=k[:, :64]), "must both be"), (dict(v=v[:3]), "must both be"),
                     (dict(v=v[0]), "must both be"), (dict(q=q[:3]), "q must have 4 rows"),
                     (dict(q=q.float()), "q must be Half"), (dict(q=q[:, :100]), "multiple of head_dim"),
                     (dict(q=None, q_out=q), "q_out needs q"), (dict(q_out=q.int()), "float32 or"),
                     (dict(q_out=q[:, 1:]), "q_out must be at least"),
                     (dict(cache=s.cache.view(torch.int8)), "cache must be torch.uint8"),
                     (dict(cache=s.cache[0]), "cache must be"), (dict(cache=s.cache[..., :64]), "cache must be"),
                     (dict(cache=s.cache.transpose(0, 1)), "contiguous pages"),
                     (dict(cache=s.cache.cpu()), "same GPU"), (dict(table=s.table.long()), "torch.int32"),
                     (dict(table=s.table[0]), "2-D"), (dict(table=s.table.cpu()), "same GPU"),
                     (dict(lens=s.lens_t[:1]), "lens must be a contiguous"),
                     (dict(lens=s.lens_t.long()), "lens must be Int"), (dict(lens=s.lens_t.cpu()), "same GPU"),
                     (dict(cu_rows=ints([0, 4])), "cu_rows must be a contiguous"),
                     (dict(freqs=f.float()), "freqs must be Double"), (dict(freqs=f.cpu()), "same GPU"),
                     (dict(positions=ints([1, 2])), "positions must be a contiguous"),
                     (dict(q_dtype=torch.bfloat16), "out_dtype")):
        with pytest.raises(ValueError, match=text):
            mq.kv_store_q4(**{**base, **kw})
    for kw, code in ((dict(k=k[:0], v=v[:0], q=q[:0]), "SHAPE"), (dict(k=k[:3], v=v[:3], q=q[:3]), "SHAPE"),
                     (dict(freqs=f[:0]), "SHAPE"), (dict(freqs=mq.rope_freqs(66, device=dev())), "SHAPE"),
                     (dict(mscale=float("inf")), "EPS"), (dict(q_out=torch.empty_like(q)), None)):
        a = {**base, **kw}
        if code is None:
            mq.kv_store_q4(**a)
            continue
        with pytest.raises(mq.MQError) as e:
            mq.kv_store_q4(**a)
        assert e.value.code == getattr(mq._lib, "MQ_ERR_" + code), kw
    x = torch.empty(4, 8 * D, dtype=torch.float16, device=dev())
    with pytest.raises(mq.MQError) as e:                 # q_out over k
        mq.kv_store_q4(x[:, :128], v, s.cache, s.table, s.lens_t, q=q, q_out=x[:, 64:320])
    assert e.value.code == mq._lib.MQ_ERR_OVERLAP
    for kw in (dict(k_out=k.int()), dict(k_out=k, v_out=v.float()), dict(k_out=k[:3]),
               dict(v_out=v[:, :100])):
        with pytest.raises(ValueError):
            mq.kv_load_q4(s.cache, s.table, s.lens_t, 4, **kw)
    with pytest.raises(mq.MQError) as e:
        mq.kv_load_q4(s.cache, s.table, s.lens_t, 4, k_out=k, v_out=k)
    assert e.value.code == mq._lib.MQ_ERR_OVERLAP
    for rows in (0, 3, -4, 1 << 40):
        with pytest.raises(mq.MQError):
            mq.kv_load_q4(s.cache, s.table, s.lens_t, rows)
