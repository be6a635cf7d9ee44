"""The C ABI of the attention operators and their Python front end, without a GPU:
every call carries exactly one defect and is refused before anything is launched."""

import ctypes
import math

import pytest
import torch

import quantized_weight_prefill_q4_amd as mq
from quantized_weight_prefill_q4_amd import _lib

FAKE = 0x100000        # 16-byte aligned, never dereferenced
Q, K, V, Y, C, T, P = (FAKE + i * 0x10000000 for i in range(7))
F32, F16 = _lib.MQ_F32, _lib.MQ_F16


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


ROPE = dict(xt=F32, X=Q, ldx=256, pos=P, freqs=T, n=64, layout=0, ms=1.0, heads=2, D=128, yt=F16,
            Y=Y, ldy=256, M=3)


def _rope(L, **kw):
    a = {**ROPE, **kw}
    return L.mq_rope(a["xt"], a["X"], a["ldx"], a["pos"], a["freqs"], a["n"], a["layout"], a["ms"],
                     a["heads"], a["D"], a["yt"], a["Y"], a["ldy"], a["M"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(X=None), _lib.MQ_ERR_NULL), (dict(pos=None), _lib.MQ_ERR_NULL),
    (dict(freqs=None), _lib.MQ_ERR_NULL), (dict(Y=None), _lib.MQ_ERR_NULL),
    (dict(xt=2), _lib.MQ_ERR_TYPE), (dict(yt=-1), _lib.MQ_ERR_TYPE),
    (dict(M=0), _lib.MQ_ERR_SHAPE), (dict(M=-4), _lib.MQ_ERR_SHAPE),
    (dict(M=(1 << 24) + 1), _lib.MQ_ERR_SHAPE), (dict(heads=0), _lib.MQ_ERR_SHAPE),
    (dict(heads=4097, ldx=1 << 20, ldy=1 << 20), _lib.MQ_ERR_SHAPE), (dict(D=0), _lib.MQ_ERR_SHAPE),
    (dict(D=1025), _lib.MQ_ERR_SHAPE), (dict(n=0), _lib.MQ_ERR_SHAPE),
    (dict(n=63), _lib.MQ_ERR_SHAPE), (dict(n=130), _lib.MQ_ERR_SHAPE),
    (dict(n=-2), _lib.MQ_ERR_SHAPE), (dict(layout=2), _lib.MQ_ERR_FORMAT),
    (dict(layout=-1), _lib.MQ_ERR_FORMAT), (dict(ms=math.nan), _lib.MQ_ERR_EPS),
    (dict(ms=math.inf), _lib.MQ_ERR_EPS), (dict(ldx=255), _lib.MQ_ERR_LD),
    (dict(ldy=255), _lib.MQ_ERR_LD), (dict(X=Q + 2), _lib.MQ_ERR_ALIGN),
    (dict(Y=Y + 1), _lib.MQ_ERR_ALIGN), (dict(pos=P + 2), _lib.MQ_ERR_ALIGN),
    (dict(freqs=T + 4), _lib.MQ_ERR_ALIGN),
    (dict(Y=Q), _lib.MQ_ERR_OVERLAP),                      # x's place in another type
    (dict(Y=Q + 4, yt=F32), _lib.MQ_ERR_OVERLAP), (dict(Y=P, yt=F32), _lib.MQ_ERR_OVERLAP),
    (dict(Y=T), _lib.MQ_ERR_OVERLAP), (dict(Y=Q, yt=F32, ldy=512), _lib.MQ_ERR_OVERLAP),
])
def test_rope_refuses(L, bad, code):
    assert _rope(L, **bad) == code


KV = dict(cache=C, page_bytes=2 * 2 * 36 * 128, pages=4, heads=2, page=64, head_dim=128, table=T,
          table_width=3, table_ld=3, lens=P, cu_rows=None, batch=2)
STORE = dict(xt=F16, K=K, ldk=256, V=V, ldv=256, freqs=T + 0x1000, n=128, layout=0, ms=1.0, pos=None,
             Q=Q, ldq=512, qh=4, qt=F16, QO=Y, ldqo=512, M=6)
ATTN = dict(xt=F16, Q=Q, ldq=512, qh=4, Y=Y, ldy=512, M=6, scale=0.1, causal=1, window=0, cap=0.0,
            slopes=None, prefix=None, max_len=192, ws=None, wsb=0)


def _kv(kw):
    a = {**KV, **{k: v for k, v in kw.items() if k in KV}}
    return ctypes.byref(_lib.MqKvQ4(**a))


def _store(L, **kw):
    a = {**STORE, **kw}
    return L.mq_kv_store_q4(_kv(kw), a["xt"], a["K"], a["ldk"], a["V"], a["ldv"], a["freqs"],
                            a["n"], a["layout"], a["ms"], a["pos"], a["Q"], a["ldq"], a["qh"],
                            a["qt"], a["QO"], a["ldqo"], a["M"], None)


def _load(L, **kw):
    a = {**STORE, **kw}
    return L.mq_kv_load_q4(_kv(kw), a["xt"], a["K"], a["ldk"], a["V"], a["ldv"], a["M"], None)


def _attn(L, **kw):
    a = {**ATTN, **kw}
    return L.mq_attention_q4(_kv(kw), a["xt"], a["Q"], a["ldq"], a["qh"], a["Y"], a["ldy"], a["M"],
                             a["scale"], a["causal"], a["window"], a["cap"], a["slopes"],
                             a["prefix"], a["max_len"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(cache=None), _lib.MQ_ERR_NULL), (dict(table=None), _lib.MQ_ERR_NULL),
    (dict(lens=None), _lib.MQ_ERR_NULL), (dict(M=0), _lib.MQ_ERR_SHAPE),
    (dict(M=5), _lib.MQ_ERR_SHAPE),                        # two sequences share no 5 rows
    (dict(head_dim=80), _lib.MQ_ERR_SHAPE), (dict(head_dim=32), _lib.MQ_ERR_SHAPE),
    (dict(head_dim=512), _lib.MQ_ERR_SHAPE), (dict(heads=0), _lib.MQ_ERR_SHAPE),
    (dict(heads=4097), _lib.MQ_ERR_SHAPE), (dict(page=48), _lib.MQ_ERR_SHAPE),
    (dict(page=0), _lib.MQ_ERR_SHAPE), (dict(page=-32), _lib.MQ_ERR_SHAPE),
    (dict(pages=0), _lib.MQ_ERR_SHAPE), (dict(batch=0), _lib.MQ_ERR_SHAPE),
    (dict(batch=-1), _lib.MQ_ERR_SHAPE), (dict(table_width=0), _lib.MQ_ERR_SHAPE),
    (dict(batch=(1 << 24) + 1, M=1 << 24), _lib.MQ_ERR_SHAPE),
    (dict(page_bytes=2 * 2 * 36 * 128 - 16), _lib.MQ_ERR_LD),
    (dict(page_bytes=2 * 2 * 36 * 128 + 8), _lib.MQ_ERR_LD), (dict(table_ld=2), _lib.MQ_ERR_LD),
    (dict(cache=C + 8), _lib.MQ_ERR_ALIGN), (dict(table=T + 2), _lib.MQ_ERR_ALIGN),
    (dict(lens=P + 1), _lib.MQ_ERR_ALIGN), (dict(cu_rows=P + 6), _lib.MQ_ERR_ALIGN),
])
def test_cache_and_batch_are_checked(L, bad, code):
    for call in (_store, _load, _attn):
        assert call(L, **bad) == code, call.__name__
    if not {"cache", "table", "lens", "cu_rows", "page_bytes", "table_ld"} & set(bad):
        a = {**ATTN, **bad}
        assert L.mq_attention_q4_workspace_bytes(_kv(bad), 4, a["M"], 192) == code
    assert L.mq_kv_store_q4(None, *[0] * 3, None, 0, None, 0, 0, 0.0, None, None, 0, 0, 0, None, 0, 6,
                            None) == _lib.MQ_ERR_NULL


@pytest.mark.parametrize("bad,code", [
    (dict(K=None), _lib.MQ_ERR_NULL), (dict(V=None), _lib.MQ_ERR_NULL),
    (dict(QO=None), _lib.MQ_ERR_NULL), (dict(xt=3), _lib.MQ_ERR_TYPE),
    (dict(qt=8), _lib.MQ_ERR_TYPE), (dict(n=130), _lib.MQ_ERR_SHAPE),
    (dict(n=0), _lib.MQ_ERR_SHAPE), (dict(layout=7), _lib.MQ_ERR_FORMAT),
    (dict(ms=-math.inf), _lib.MQ_ERR_EPS), (dict(qh=0), _lib.MQ_ERR_SHAPE),
    (dict(ldk=255), _lib.MQ_ERR_LD), (dict(ldv=255), _lib.MQ_ERR_LD),
    (dict(ldq=511), _lib.MQ_ERR_LD), (dict(ldqo=511), _lib.MQ_ERR_LD),
    (dict(K=K + 1), _lib.MQ_ERR_ALIGN), (dict(V=V + 1), _lib.MQ_ERR_ALIGN),
    (dict(QO=Y + 1), _lib.MQ_ERR_ALIGN), (dict(pos=P + 2), _lib.MQ_ERR_ALIGN),
    (dict(freqs=T + 4), _lib.MQ_ERR_ALIGN),
    (dict(K=C + 64), _lib.MQ_ERR_OVERLAP), (dict(V=C + 4 * 18432 - 2), _lib.MQ_ERR_OVERLAP),
    (dict(QO=C), _lib.MQ_ERR_OVERLAP), (dict(QO=K), _lib.MQ_ERR_OVERLAP),
    (dict(QO=V), _lib.MQ_ERR_OVERLAP), (dict(Q=C), _lib.MQ_ERR_OVERLAP),
    (dict(QO=Q, qt=F32, ldqo=512), _lib.MQ_ERR_OVERLAP), (dict(QO=Q + 2), _lib.MQ_ERR_OVERLAP),
])
def test_store_refuses(L, bad, code):
    assert _store(L, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(K=None), _lib.MQ_ERR_NULL), (dict(V=None), _lib.MQ_ERR_NULL),
    (dict(xt=24), _lib.MQ_ERR_TYPE), (dict(ldk=255), _lib.MQ_ERR_LD),
    (dict(ldv=0), _lib.MQ_ERR_LD), (dict(K=K + 1), _lib.MQ_ERR_ALIGN),
    (dict(V=V + 1), _lib.MQ_ERR_ALIGN), (dict(V=K), _lib.MQ_ERR_OVERLAP),
    (dict(K=C), _lib.MQ_ERR_OVERLAP), (dict(V=C + 2), _lib.MQ_ERR_OVERLAP),
])
def test_load_refuses(L, bad, code):
    assert _load(L, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(Q=None), _lib.MQ_ERR_NULL), (dict(Y=None), _lib.MQ_ERR_NULL), (dict(xt=9), _lib.MQ_ERR_TYPE),
    (dict(qh=3), _lib.MQ_ERR_SHAPE), (dict(qh=0), _lib.MQ_ERR_SHAPE),
    (dict(qh=-2), _lib.MQ_ERR_SHAPE), (dict(max_len=-1), _lib.MQ_ERR_SHAPE),
    (dict(scale=math.nan), _lib.MQ_ERR_EPS), (dict(scale=math.inf), _lib.MQ_ERR_EPS),
    (dict(cap=-1.0), _lib.MQ_ERR_EPS), (dict(cap=math.nan), _lib.MQ_ERR_EPS),
    (dict(cap=math.inf), _lib.MQ_ERR_EPS), (dict(window=-1), _lib.MQ_ERR_EPS),
    (dict(ldq=511), _lib.MQ_ERR_LD), (dict(ldy=511), _lib.MQ_ERR_LD),
    (dict(Q=Q + 1), _lib.MQ_ERR_ALIGN), (dict(Y=Y + 1), _lib.MQ_ERR_ALIGN),
    (dict(slopes=P + 2), _lib.MQ_ERR_ALIGN), (dict(prefix=P + 2), _lib.MQ_ERR_ALIGN),
    (dict(Y=Q), _lib.MQ_ERR_OVERLAP), (dict(Y=C), _lib.MQ_ERR_OVERLAP),
    (dict(table_width=400, table_ld=400, max_len=25600), _lib.MQ_ERR_WORKSPACE),
    (dict(table_width=400, table_ld=400, max_len=25600, ws=K + 4, wsb=1 << 40),
     _lib.MQ_ERR_WORKSPACE),
    (dict(table_width=400, table_ld=400, max_len=25600, ws=K, wsb=64), _lib.MQ_ERR_WORKSPACE),
    (dict(table_width=400, table_ld=400, max_len=25600, ws=Q, wsb=1 << 40), _lib.MQ_ERR_OVERLAP),
    (dict(table_width=400, table_ld=400, max_len=25600, ws=Y, wsb=1 << 40), _lib.MQ_ERR_OVERLAP),
    (dict(table_width=400, table_ld=400, max_len=25600, ws=C, wsb=1 << 40), _lib.MQ_ERR_OVERLAP),
])
def test_attention_refuses(L, bad, code):
    assert _attn(L, **bad) == code


LIST = K + 0x8000000       # of the call's lists, where a test gives one a place of its own


@pytest.mark.parametrize("name", ["table", "lens", "cu_rows", "pos", "freqs", "slopes", "prefix"])
def test_outputs_over_a_list_of_the_call_are_refused(L, name):
    """An output may not overlap what the kernels read beside it: the lists that say where rows
    and tokens are, positions, frequencies, slopes and prefixes.  By its last element too."""
    size = {"table": 2 * 3 * 4, "lens": 8, "cu_rows": 12, "pos": 24, "freqs": 512, "slopes": 16,
            "prefix": 8}[name]
    lists = {name: LIST}
    end = LIST + size
    plan = dict(table_width=3, max_len=1 << 20)
    ws = dict(wsb=1 << 40, Y=Y, **plan)
    row = 6 * 512 * 2                                   # bytes of a Q, QO or Y of M rows
    if name not in ("slopes", "prefix"):
        for qo in (LIST, end - 4 - end % 2, LIST - row + 4):
            assert _store(L, QO=qo, **lists) == _lib.MQ_ERR_OVERLAP, hex(qo)
        for c in (LIST, (end - 1) & ~15, LIST + 16 - 4 * 18432):
            assert _store(L, cache=c, Q=None, **lists) == _lib.MQ_ERR_OVERLAP, hex(c)
    if name in ("table", "lens", "cu_rows"):
        for p in (LIST, end - 4, LIST - 6 * 256 * 2 + 4):
            assert _load(L, K=p, V=V, **lists) == _lib.MQ_ERR_OVERLAP
            assert _load(L, K=Y, V=p, **lists) == _lib.MQ_ERR_OVERLAP
    if name not in ("pos", "freqs"):
        for y in (LIST, end - 4, LIST - row + 4):
            assert _attn(L, Y=y, **lists) == _lib.MQ_ERR_OVERLAP
        need = L.mq_attention_q4_workspace_bytes(_kv(plan), 4, 6, 1 << 20)
        assert need > 0
        for w in (LIST, (end - 1) & ~15, LIST + 16 - need):
            assert _attn(L, ws=w, **ws, **lists) == _lib.MQ_ERR_OVERLAP


def test_sizes(L):
    assert mq.kv_page_bytes(8, 64, 128) == 8 * 2 * 36 * 128
    for bad in ((0, 64, 128), (8, 33, 128), (8, 64, 100), (1 << 32, 64, 128)):
        with pytest.raises(mq.MQError) as e:
            mq.kv_page_bytes(*bad)
        assert e.value.code == _lib.MQ_ERR_SHAPE
    c = mq.kv_cache_q4(3, 2, 64, 96, device="cpu")
    assert c.shape == (3, 2, 2, 36 * 96) and c.dtype == torch.uint8
    # one short sequence needs no workspace, a long one parts of (D + 2) floats a row
    assert mq.attention_workspace_bytes(c, 1, 4, 1, 64) == 0
    for ragged in (False, True):
        assert mq.attention_workspace_bytes(c, 2, 4, 2, 100000, ragged) % (98 * 4 * 16) == 0
        assert mq.attention_workspace_bytes(c, 2, 4, 2, 100000, ragged) > 0
    with pytest.raises(mq.MQError):
        mq.attention_workspace_bytes(c, 2, 4, 3, 64)
    with pytest.raises(mq.MQError):
        mq.attention_workspace_bytes(c, 2, 3, 2, 64)
    with pytest.raises(ValueError):
        mq.attention_workspace_bytes(c[0], 2, 4, 2, 64)


def test_frequencies():
    f = mq.rope_freqs(8, 10000.0)
    assert f.dtype == torch.float64 and torch.allclose(
        f, torch.tensor([1, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    assert torch.equal(mq.rope_freqs(8, scale=4.0), f / 4)
    assert torch.allclose(mq.rope_freqs(8, factors=[1, 2, 4, 8]),
                          f / torch.tensor([1, 2, 4, 8], dtype=torch.float64), rtol=1e-15)
    # by parts: of 1000 positions the pairs turn 159, 15.9, 1.59 and 0.159 times
    g = mq.rope_freqs(8, scale=4.0, context=1000)
    w = [1.0, (100 / (2 * math.pi) - 1) / 31, (10 / (2 * math.pi) - 1) / 31, 0.0]
    for j in range(4):
        assert math.isclose(float(g[j]), float(f[j]) * (w[j] + (1 - w[j]) / 4), rel_tol=1e-13)
    for bad in (dict(n_rot=7), dict(n_rot=0), dict(n_rot=8, base=0.0), dict(n_rot=8, scale=-1.0),
                dict(n_rot=8, base=math.nan), dict(n_rot=8, factors=[1, 2]),
                dict(n_rot=8, context=100, beta=(3.0, 3.0))):
        with pytest.raises(ValueError):
            mq.rope_freqs(**bad)


def test_front_end_refuses_without_a_gpu():
    """Host tensors and unknown names are refused before the library is called."""
    x, p, f = torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), mq.rope_freqs(64)
    c, t = mq.kv_cache_q4(2, 1, 32, 64, device="cpu"), torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="unknown layout"):
        mq.rope(x, p, f, 64, layout="quarter")
    with pytest.raises(ValueError, match="unknown layout"):
        mq.kv_store_q4(x, x, c, t, p, layout=None)
    with pytest.raises(ValueError, match="out_dtype"):
        mq.rope(x, p, f, 64, out_dtype=torch.bfloat16)
    for call in (lambda: mq.rope(x, p, f, 64), lambda: mq.kv_store_q4(x, x, c, t, p),
                 lambda: mq.kv_load_q4(c, t, p, 2), lambda: mq.attention_q4(x, c, t, p)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
