"""Sizes and strides that do not fit the C ABI's int are refused by the Python
front end (ctypes would pass their low 32 bits).  No GPU and no memory: the
matrices are meta tensors."""

import pytest
import torch

import quantized_weight_prefill_q4_amd as mq
from quantized_weight_prefill_q4_amd import _lib, api

WRAPS = 1 << 32          # + n has the low 32 bits of n


def _rows(n, k, stride):
    return torch.empty_strided((n, k), (stride, 1), device="meta")


@pytest.mark.parametrize("stride", [1 << 31, WRAPS, WRAPS + 64])
def test_row_strides(stride):
    with pytest.raises(ValueError, match="elements apart"):
        api._row_major_2d(_rows(2, 64, stride), "x")
    one = api._row_major_2d(_rows(1, 64, stride), "x")     # a single row has no stride
    assert 64 <= one <= api._INT_MAX


def test_strides_that_fit():
    for stride in (64, (1 << 31) - 1):
        assert api._row_major_2d(_rows(2, 64, stride), "x") == stride


def test_sizes_of_matrices():
    big = torch.empty_strided((WRAPS + 40, 8), (8, 1), device="meta")
    for rows, cols in ((WRAPS + 40, 8), (40, WRAPS + 8)):
        with pytest.raises(mq.MQError) as e:
            api._need_shape(big, rows, cols, "x")
        assert e.value.code == _lib.MQ_ERR_SHAPE
    api._need_shape(big, 40, 8, "x")


@pytest.mark.parametrize("query", [
    lambda *a: mq.workspace_bytes(0, *a), lambda *a: mq.workspace_bytes("q4_k", *a, x_f32=True),
    lambda *a: mq.mmq_workspace_bytes("q4_k", *a),
    lambda *a: mq.linear_workspace_bytes(0, *a), lambda *a: mq.linear_workspace_bytes("q4_k", *a),
    lambda *a: mq.linear_workspace_bytes(0, *a, glu=True), lambda *a: mq.gemm_plan(0, *a),
    lambda *a: mq.gemm_plan("q4_k", *a, path="mmq")])
def test_queries(query):
    size = [40, 512, 512, 2]
    query(*size)
    for i in range(4):
        for wrap in (WRAPS, -WRAPS):
            bad = list(size)
            bad[i] += wrap
            with pytest.raises(mq.MQError) as e:
                query(*bad)
            assert e.value.code == (_lib.MQ_ERR_SPLIT if i == 3 else _lib.MQ_ERR_SHAPE)


def test_bounds_of_lengths():
    """max_len is 64 bits wide: what does not fit is refused by the size query as by the call."""
    c = mq.kv_cache_q4(3, 2, 64, 128, device="cpu")
    need = mq.attention_workspace_bytes(c, 1, 4, 1, 1 << 30)
    assert need > 0
    for fits in ((1 << 30) + 1, WRAPS, (1 << 63) - 1):
        assert mq.attention_workspace_bytes(c, 1, 4, 1, fits) == need
    for wraps in (1 << 63, 1 << 64, (1 << 64) + 40, -(1 << 64) + 40):
        with pytest.raises(OverflowError):
            mq.attention_workspace_bytes(c, 1, 4, 1, wraps)
    for bad in (40.0, None, "40"):
        with pytest.raises(TypeError):
            mq.attention_workspace_bytes(c, 1, 4, 1, bad)
    for neg in (-1, -(1 << 63)):
        with pytest.raises(mq.MQError) as e:
            mq.attention_workspace_bytes(c, 1, 4, 1, neg)
        assert e.value.code == _lib.MQ_ERR_SHAPE


def test_formats():
    for fmt in (WRAPS + _lib.MQ_Q4_K, _lib.MQ_Q4_K - WRAPS):
        for query in (lambda: mq.row_bytes(fmt, 256), lambda: mq.block_bytes(fmt),
                      lambda: mq.workspace_bytes(fmt, 40, 512, 512),
                      lambda: mq.linear_workspace_bytes(fmt, 40, 512, 512)):
            with pytest.raises(mq.MQError) as e:
                query()
            assert e.value.code == _lib.MQ_ERR_FORMAT
    assert mq.row_bytes(_lib.MQ_Q4_K, 256) == 144
