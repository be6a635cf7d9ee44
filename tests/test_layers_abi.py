"""The C ABI of the operators around the quantized products, without a GPU:
every call below carries exactly one defect and is refused before anything is
launched."""

import pytest

from quantized_weight_prefill_q4_amd import _lib

FAKE = 0x100000        # 16-byte aligned, never dereferenced
R, W, H, Y, D = (FAKE + i * 0x1000000 for i in range(1, 6))
F32, F16 = _lib.MQ_F32, _lib.MQ_F16


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


NORM = dict(xt=F32, X=FAKE, ldx=64, rt=F32, R=R, ldr=64, w=W, eps=1e-6, H=H, ldh=64, yt=F16, Y=Y,
            ldy=64, M=4, K=64)


def _norm(L, **kw):
    a = {**NORM, **kw}
    return L.mq_add_rms_norm(a["xt"], a["X"], a["ldx"], a["rt"], a["R"], a["ldr"], a["w"], a["eps"],
                             a["H"], a["ldh"], a["yt"], a["Y"], a["ldy"], a["M"], a["K"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(X=None), _lib.MQ_ERR_NULL), (dict(w=None), _lib.MQ_ERR_NULL),
    (dict(H=None), _lib.MQ_ERR_NULL), (dict(Y=None), _lib.MQ_ERR_NULL),
    (dict(xt=2), _lib.MQ_ERR_TYPE), (dict(rt=-1), _lib.MQ_ERR_TYPE), (dict(yt=8), _lib.MQ_ERR_TYPE),
    (dict(M=0), _lib.MQ_ERR_SHAPE), (dict(K=0), _lib.MQ_ERR_SHAPE),
    (dict(M=(1 << 24) + 1), _lib.MQ_ERR_SHAPE), (dict(K=-5), _lib.MQ_ERR_SHAPE),
    (dict(ldx=63), _lib.MQ_ERR_LD), (dict(ldr=0), _lib.MQ_ERR_LD), (dict(ldh=63), _lib.MQ_ERR_LD),
    (dict(ldy=63), _lib.MQ_ERR_LD),
    (dict(X=FAKE + 2), _lib.MQ_ERR_ALIGN), (dict(Y=Y + 1), _lib.MQ_ERR_ALIGN),
    (dict(w=W + 2), _lib.MQ_ERR_ALIGN), (dict(R=R + 1), _lib.MQ_ERR_ALIGN),
    (dict(H=H + 2), _lib.MQ_ERR_ALIGN),
    (dict(eps=-1e-9), _lib.MQ_ERR_EPS), (dict(eps=float("nan")), _lib.MQ_ERR_EPS),
    (dict(eps=float("inf")), _lib.MQ_ERR_EPS),
    (dict(H=R + 4), _lib.MQ_ERR_OVERLAP),               # the stream, shifted by one element
    (dict(Y=H, yt=F32), _lib.MQ_ERR_OVERLAP),           # one buffer for both outputs
    (dict(Y=FAKE), _lib.MQ_ERR_OVERLAP),                # x's place in another type
    (dict(Y=W, M=1), _lib.MQ_ERR_OVERLAP),
    (dict(H=FAKE, ldh=128), _lib.MQ_ERR_OVERLAP),       # x's place at another stride
    (dict(X=FAKE, ldx=128, Y=FAKE + 63 * 4, yt=F32, ldy=128), _lib.MQ_ERR_OVERLAP),
])
def test_norm_refuses(L, bad, code):
    assert _norm(L, **bad) == code


def _norm_q8(L, **kw):
    a = {**NORM, "ds": D, **kw}
    return L.mq_add_rms_norm_q8_1(a["xt"], a["X"], a["ldx"], a["rt"], a["R"], a["ldr"], a["w"],
                                  a["eps"], a["H"], a["ldh"], a["Y"], a["ldy"], a["ds"], a["M"],
                                  a["K"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(Y=None), _lib.MQ_ERR_NULL), (dict(ds=None), _lib.MQ_ERR_NULL),
    (dict(X=None), _lib.MQ_ERR_NULL), (dict(xt=7), _lib.MQ_ERR_TYPE),
    (dict(K=48), _lib.MQ_ERR_SHAPE), (dict(ldy=72), _lib.MQ_ERR_LD), (dict(ldy=48), _lib.MQ_ERR_LD),
    (dict(Y=Y + 8), _lib.MQ_ERR_ALIGN), (dict(ds=D + 8), _lib.MQ_ERR_ALIGN),
    (dict(eps=-1.0), _lib.MQ_ERR_EPS), (dict(Y=FAKE), _lib.MQ_ERR_OVERLAP),
    (dict(ds=Y + 64), _lib.MQ_ERR_OVERLAP), (dict(ds=H), _lib.MQ_ERR_OVERLAP),
])
def test_norm_q8_1_refuses(L, bad, code):
    assert _norm_q8(L, **bad) == code


def test_error_texts(L):
    known = {L.mq_strerror(c) for c in range(_lib.MQ_ERR_OVERLAP, 1)}
    assert len(known) == 1 - _lib.MQ_ERR_OVERLAP and b"unknown error code" not in known
