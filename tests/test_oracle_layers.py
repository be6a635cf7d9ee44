"""The layers oracle against hand-derived values (CPU)."""

import math
import os
import re

import numpy as np
import pytest

from conftest import ROOT
from oracle import layers


def test_rms_norm_worked_row():
    # h = (3, -4): mean of squares 12.5; with eps 0 the norm is h / sqrt(12.5)
    y, h = layers.rms_norm_ref(np.array([[1.0, -3.0]]), np.array([1.0, 2.0]), 0.0,
                               np.array([[2.0, -1.0]], dtype=np.float32))
    assert h.tolist() == [[3.0, -4.0]]
    assert np.allclose(y, [[3 / math.sqrt(12.5), -8 / math.sqrt(12.5)]], rtol=1e-15)
    y, h = layers.rms_norm_ref(np.zeros((1, 4)), np.ones(4), 1e-6)
    assert not y.any() and not h.any()


def test_stream_is_rounded_to_its_type():
    # 2048 + 1 is not an f16 value (step 2 there): ties to even gives 2048
    _, h = layers.rms_norm_ref(np.array([[1.0]]), np.ones(1), 0.0,
                               np.array([[2048.0]], dtype=np.float16))
    assert h[0, 0] == 2048.0


@pytest.mark.parametrize("act,at1", [("none", 1.0), ("relu", 1.0), ("silu", 1 / (1 + math.exp(-1))),
                                     ("gelu", 0.5 * (1 + math.erf(1 / math.sqrt(2)))),
                                     ("gelu_tanh", 0.5 * (1 + math.tanh(math.sqrt(2 / math.pi)
                                                                         * 1.044715)))])
def test_activations_at_one_and_far_away(act, at1):
    v = layers.act_ref(np.array([1.0, 0.0, 50.0, -50.0]), act)
    assert v[0] == pytest.approx(at1, rel=1e-14) and v[1] == 0.0
    assert v[2] == pytest.approx(50.0, rel=1e-15)
    assert v[3] == (-50.0 if act == "none" else pytest.approx(0.0, abs=1e-19))


def test_glu_halves():
    x = np.array([[1.0, 2.0]], dtype=np.float16).view(np.uint16)
    w = np.array([[1, 0], [0, 1], [3, 0], [0, 3]], dtype=np.float16).view(np.uint16)
    y, g, u, sg, su = layers.glu_ref(x, w, 2, bias=np.array([0.0, 0, 1, 1]), act="relu")
    assert g.tolist() == [[1, 2]] and u.tolist() == [[4, 7]] and y.tolist() == [[4, 14]]
    y, S = layers.linear_ref(x, w, 2, bias=np.array([-5.0, 0, 0, 0]), act="relu",
                             residual=np.ones((1, 4)))
    assert y.tolist() == [[1, 3, 4, 7]] and S.tolist() == [[6, 2, 3, 6]]


def test_gelu_polynomial():
    """The kernels' polynomial for h = 0.5·e^(z²)·erfc(z), its coefficients read
    from the source, over the z it is used for: the fit's error with the f32
    coefficients as stored, and that of its evaluation in f32.  The latter, in
    units of 2^-24 of h and largest towards z = 0, where t = -1 and h = 0.5: a
    rounding of each of the eleven partial sums, which add up to 1.35 there (2.7
    of h), and three roundings in t, with |dh/dt · t| = 0.85 (5.1 of h): 8."""
    src = open(os.path.join(ROOT, "quantized_weight_prefill_q4_amd", "csrc", "epilogue.h")).read()
    body = src[src.index("float gelu_f32(float v)"):]
    body = body[:body.index("return")]
    coeffs = re.findall(r"float h = ([-+.e0-9]+)f;", body)
    coeffs += re.findall(r"fmaf\(h, t, ([-+.e0-9]+)f\)", body)
    coeffs = np.array(coeffs, dtype=np.float64).astype(np.float32)
    assert len(coeffs) == 11
    z = np.linspace(0, 9, 9001).astype(np.float32)
    ref = np.array([0.5 * math.exp(v * v) * math.erfc(v) for v in z.astype(np.float64)])
    h, t = np.zeros(len(z)), (z.astype(np.float64) - 3) / (z.astype(np.float64) + 3)
    for c in coeffs.astype(np.float64):
        h = h * t + c
    assert np.max(np.abs(h / ref - 1)) <= 1.25e-8
    t = (z - np.float32(3)) / (z + np.float32(3))
    h = np.zeros(len(z), np.float32)
    for c in coeffs:   # a fused multiply-add: one rounding
        h = (h.astype(np.float64) * t.astype(np.float64) + np.float64(c)).astype(np.float32)
    assert np.max(np.abs(h / ref - 1)) <= 8 * 2.0 ** -24
