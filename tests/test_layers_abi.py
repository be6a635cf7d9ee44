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


LIN = dict(xt=F16, X=FAKE, ldx=512, W=W, ldw=512, b=H, act=2, rt=F32, R=R, ldr=96, yt=F32, Y=Y,
           ldy=96, M=300, N=96, K=512, ws=None, wsb=0, split=1)


def _linear(L, fmt=0, **kw):
    a = {**LIN, **kw}
    w = (a["W"], a["ldw"]) if fmt == 0 else (fmt, a["W"])
    f = L.mq_linear_f16cache if fmt == 0 else L.mq_linear_fused
    return f(a["xt"], a["X"], a["ldx"], *w, a["b"], a["act"], a["rt"], a["R"], a["ldr"], a["yt"],
             a["Y"], a["ldy"], a["M"], a["N"], a["K"], a["ws"], a["wsb"], a["split"], None)


def _glu(L, fmt=0, **kw):
    a = {**LIN, **kw}
    w = (a["W"], a["ldw"]) if fmt == 0 else (fmt, a["W"])
    f = L.mq_glu_f16cache if fmt == 0 else L.mq_glu_fused
    return f(a["xt"], a["X"], a["ldx"], *w, a["b"], a["act"], a["yt"], a["Y"], a["ldy"], a["M"],
             a["N"], a["K"], a["ws"], a["wsb"], a["split"], None)


LAYER_BAD = [
    (dict(X=None), _lib.MQ_ERR_NULL), (dict(W=None), _lib.MQ_ERR_NULL),
    (dict(Y=None), _lib.MQ_ERR_NULL),
    (dict(xt=2), _lib.MQ_ERR_TYPE), (dict(yt=-1), _lib.MQ_ERR_TYPE),
    (dict(act=5), _lib.MQ_ERR_ACT), (dict(act=-1), _lib.MQ_ERR_ACT),
    (dict(M=0), _lib.MQ_ERR_SHAPE), (dict(N=0), _lib.MQ_ERR_SHAPE),
    (dict(N=-(1 << 31)), _lib.MQ_ERR_SHAPE), (dict(N=(1 << 31) - 1), _lib.MQ_ERR_SHAPE),
    (dict(K=500), _lib.MQ_ERR_SHAPE), (dict(K=0), _lib.MQ_ERR_SHAPE),
    (dict(ldx=508), _lib.MQ_ERR_LD), (dict(ldx=504), _lib.MQ_ERR_LD),
    (dict(xt=F32, ldx=514, ws=D, wsb=1 << 30), _lib.MQ_ERR_LD),
    (dict(ldy=95), _lib.MQ_ERR_LD),
    (dict(X=FAKE + 8), _lib.MQ_ERR_ALIGN), (dict(W=W + 2), _lib.MQ_ERR_ALIGN),
    (dict(Y=Y + 2), _lib.MQ_ERR_ALIGN), (dict(b=H + 2), _lib.MQ_ERR_ALIGN),
    (dict(split=17), _lib.MQ_ERR_SPLIT), (dict(split=-1), _lib.MQ_ERR_SPLIT),
    (dict(split=4), _lib.MQ_ERR_WORKSPACE),
    (dict(split=4, ws=D, wsb=100), _lib.MQ_ERR_WORKSPACE),
    (dict(split=4, ws=D + 8, wsb=1 << 30), _lib.MQ_ERR_WORKSPACE),
    (dict(split=4, ws=Y + 64, wsb=1 << 30), _lib.MQ_ERR_OVERLAP),
    (dict(split=4, ws=FAKE + 1024, wsb=1 << 30), _lib.MQ_ERR_OVERLAP),
    (dict(split=4, ws=W + 1024, wsb=1 << 30), _lib.MQ_ERR_OVERLAP),
    (dict(split=4, ws=H, wsb=1 << 30), _lib.MQ_ERR_OVERLAP),
    (dict(Y=FAKE, ldx=512, ldy=96), _lib.MQ_ERR_OVERLAP),      # x's place
    (dict(Y=W), _lib.MQ_ERR_OVERLAP), (dict(Y=H), _lib.MQ_ERR_OVERLAP),
]


@pytest.mark.parametrize("bad,code", LAYER_BAD + [
    (dict(ldw=520 + 4), _lib.MQ_ERR_LD), (dict(ldw=504), _lib.MQ_ERR_LD)])
def test_f16cache_layers_refuse(L, bad, code):
    assert _linear(L, **bad) == code
    assert _glu(L, **bad) == code


@pytest.mark.parametrize("bad,code", LAYER_BAD + [(dict(K=384), _lib.MQ_ERR_SHAPE)])
@pytest.mark.parametrize("fmt", [12, 14])
def test_fused_layers_refuse(L, fmt, bad, code):
    assert _linear(L, fmt, **bad) == code
    assert _glu(L, fmt, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(rt=3), _lib.MQ_ERR_TYPE), (dict(ldr=95), _lib.MQ_ERR_LD),
    (dict(R=R + 2), _lib.MQ_ERR_ALIGN),
    (dict(R=Y + 4), _lib.MQ_ERR_OVERLAP),               # the stream, shifted
    (dict(R=Y, rt=F16), _lib.MQ_ERR_OVERLAP),           # in another type
    (dict(R=Y, ldr=104), _lib.MQ_ERR_OVERLAP),          # at another stride
])
def test_residuals_refused(L, bad, code):
    assert _linear(L, **bad) == code and _linear(L, 12, **bad) == code


def test_short_k_is_not_split_over_many_tiles(L):
    assert L.mq_gemm_workspace_bytes(0, 512, 2048, 512, 0) > 0
    assert L.mq_linear_workspace_bytes(0, F16, 512, 2048, 512, 0) == 0
    assert L.mq_glu_workspace_bytes(0, F16, 512, 1024, 512, 0) == 0
    assert L.mq_linear_workspace_bytes(0, F16, 512, 2048, 512, 2) > 0        # asked for
    assert L.mq_linear_workspace_bytes(0, F16, 512, 2048, 1032, 0) > 0


def test_few_rows_need_no_workspace(L):
    for xt in (F16, F32):
        for M in (1, 4, 16):
            assert L.mq_linear_workspace_bytes(0, xt, M, 3584, 18944, 0) == 0
            assert L.mq_glu_workspace_bytes(14, xt, M, 14336, 4096, 0) == 0
        assert L.mq_linear_workspace_bytes(12, xt, 32, 14336, 4096, 0) == 0
        assert L.mq_linear_workspace_bytes(0, xt, 32, 3584, 3584, 0) == 0
    # a split asked for is the tile kernel's, at any M
    assert L.mq_linear_workspace_bytes(0, F16, 1, 128, 512, 2) == 2 * 64 * 128 * 4
    # from 17 rows on a large f16 cache takes the tile kernel, too
    assert L.mq_linear_workspace_bytes(0, F16, 17, 3584, 18944, 0) == \
        L.mq_gemm_workspace_bytes(0, 17, 3584, 18944, 0) > 0


def test_unknown_formats(L):
    for fmt in (1, 5, 99, -1):
        for f in (L.mq_linear_fused, L.mq_glu_fused):
            n = 19 if f is L.mq_linear_fused else 16
            assert f(*([F16, FAKE, 512, fmt, W] + [0] * (n - 5) + [None])) == _lib.MQ_ERR_FORMAT
        assert L.mq_linear_workspace_bytes(fmt, F16, 1, 64, 256, 0) == _lib.MQ_ERR_FORMAT
    assert L.mq_linear_fused(F16, FAKE, 512, 0, W, None, 0, 0, None, 0, F32, Y, 96, 4, 96, 512,
                             None, 0, 0, None) == _lib.MQ_ERR_FORMAT
    assert L.mq_glu_workspace_bytes(12, 9, 1, 64, 256, 0) == _lib.MQ_ERR_TYPE
    assert L.mq_glu_workspace_bytes(12, F16, 1, (1 << 23) + 1, 256, 0) == _lib.MQ_ERR_SHAPE


def test_layer_workspaces(L):
    """The planes of the matching product, after the converted f32 activations."""
    for M, N, K in ((2048, 3584, 18944), (300, 96, 512), (2048, 512, 3584)):
        planes = L.mq_gemm_workspace_bytes(0, M, N, K, 0)
        assert L.mq_linear_workspace_bytes(0, F16, M, N, K, 0) == planes
        x16 = (M * (K + (64 if K % 1024 == 0 else 0)) * 2 + 255) // 256 * 256
        assert L.mq_linear_workspace_bytes(0, F32, M, N, K, 0) == x16 + planes
        assert L.mq_glu_workspace_bytes(12, F16, M, N, 3584, 0) == \
            L.mq_gemm_workspace_bytes(12, M, 2 * N, 3584, 0)


def test_native_binding_refuses_without_a_gpu():
    """The native side's own checks: CPU tensors, non-tensors, wrong counts."""
    import torch

    import quantized_weight_prefill_q4_amd as mq
    from quantized_weight_prefill_q4_amd import layers

    b = layers._binding()
    x, w = torch.zeros(2, 32), torch.zeros(32)
    for call, args in ((b.norm, (0, x, w, None, 1e-6, 0, None, None, None)),
                       (b.layer, (0, x, w, 0, -1, -1, None, 0, None, False, 0, 0, None, None))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call(*args)
        with pytest.raises(ValueError, match="x must be a tensor"):
            call(0, 7, *args[2:])
        with pytest.raises(TypeError, match="arguments"):
            call(*args[:-1])
        with pytest.raises(TypeError):
            call("stream", *args[1:])
    with pytest.raises(ValueError, match="missing"):
        b.bind({})
    layers._binding.cache_clear()
    layers._binding()                                   # bound again
    for f, args in ((mq.add_rms_norm, (x, w)), (mq.add_rms_norm_q8_1, (x, w)),
                    (mq.linear_f16cache, (x, x.half())), (mq.glu_f16cache, (x, x.half())),
                    (mq.linear_fused, (x, x, "q8_0", 2)), (mq.glu_fused, (x, x, "q8_0", 1))):
        with pytest.raises(ValueError, match="GPU tensor"):
            f(*args)
    with pytest.raises(ValueError, match="unknown activation"):
        mq.linear_f16cache(x, x.half(), act="swish")
    with pytest.raises(ValueError, match="out_dtype"):
        mq.add_rms_norm(x, w, out_dtype=torch.bfloat16)


def test_native_binding_refuses_strides_beyond_int():
    """Rows further apart than the C ABI's int can say: of x, before its device is
    looked at (meta tensors have strides without memory)."""
    import torch

    from quantized_weight_prefill_q4_amd import layers

    b = layers._binding()
    w = torch.zeros(32)
    for stride in (1 << 31, (1 << 32) + 32):
        x = torch.empty_strided((2, 32), (stride, 1), device="meta", dtype=torch.float16)
        for call, args in ((b.norm, (x, w, None, 1e-6, 0, None, None, None)),
                           (b.layer, (x, w, 0, -1, -1, None, 0, None, False, 0, 0, None, None))):
            with pytest.raises(ValueError, match="elements apart"):
                call(0, *args)
    # one row has no stride, and the largest int is one
    for shape, stride in (((1, 32), 1 << 31), ((2, 32), (1 << 31) - 1)):
        x = torch.empty_strided(shape, (stride, 1), device="meta", dtype=torch.float16)
        with pytest.raises(ValueError, match="GPU tensor"):
            b.norm(0, x, w, None, 1e-6, 0, None, None, None)


def test_every_error_has_its_text(L):
    """All codes of the ABI, the last ones included."""
    codes = range(_lib.MQ_ERR_ACT, 1)
    assert min(v for k, v in vars(_lib).items() if k.startswith("MQ_ERR_")) == _lib.MQ_ERR_ACT
    texts = [L.mq_strerror(c) for c in codes]
    assert len(set(texts)) == len(codes) and b"unknown error code" not in texts
    assert L.mq_strerror(_lib.MQ_ERR_ACT - 1) == b"unknown error code"
