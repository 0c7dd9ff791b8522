"""The 64-bit forms of the routing rules and 8-bit products, pinned by hand."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import route_i8_oracle as orc
from quantized_moe_decode_affine_amd import synth


def test_sigmoid_bias_moves_the_choice_and_not_the_weight():
    l = np.array([[0.0, 1.0, -1.0, 2.0]])
    s = 1 / (1 + np.exp(-l[0]))
    ids, w = orc.route_rule(l, 2, "sigmoid", bias=[0.9, 0, 0, 0], renormalise=False, scale=2.0)
    assert ids.tolist() == [[0, 3]]                       # 0.5 + 0.9 before sigmoid(2)
    np.testing.assert_allclose(w, [[2 * s[0], 2 * s[3]]])
    ids, w = orc.route_rule(l, 2, "sigmoid", bias=[0.9, 0, 0, 0])
    np.testing.assert_allclose(w, [[s[0] / (s[0] + s[3]), s[3] / (s[0] + s[3])]])


def test_groups_by_one_and_by_two_terms():
    l = np.log(np.array([[5.0, 1.0, 3.0, 3.0, 2.0, 2.0]]))     # softmax: 5/16 1/16 | 3/16 3/16 | 2/16 2/16
    assert orc.route_rule(l, 2, n_groups=3, top_groups=1, group_terms=1)[0].tolist() == [[0, 1]]
    # 5 + 1 = 3 + 3 up to rounding of the logs: take a clear case
    l = np.log(np.array([[5.0, 0.5, 3.0, 3.0, 2.0, 2.0]]))
    assert orc.route_rule(l, 2, n_groups=3, top_groups=1, group_terms=2)[0].tolist() == [[2, 3]]
    assert orc.route_rule(l, 3, n_groups=3, top_groups=2, group_terms=2)[0].tolist() == [[0, 2, 3]]


def test_ties_and_closed_experts():
    l = np.zeros((1, 6))
    assert orc.route_rule(l, 3, "sigmoid", n_groups=3, top_groups=2)[0].tolist() == [[0, 1, 2]]
    l[0, [0, 3]] = -np.inf, np.nan
    ids, w = orc.route_rule(l, 5, bias=[0, -np.inf, 0, 0, 0, 0])
    assert ids.tolist() == [[2, 4, 5, -1, -1]]
    np.testing.assert_allclose(w, [[1 / 3, 1 / 3, 1 / 3, 0, 0]])
    assert orc.route_rule(np.full((1, 4), -np.inf), 2)[0].tolist() == [[-1, -1]]


def test_quantize_against_rationals():
    rng = np.random.default_rng(3)
    bits = np.concatenate([synth.to_bf16_bits(rng.standard_normal((6, 64)).astype(np.float32)),
                           synth.to_bf16_bits(np.arange(-32, 32, dtype=np.float32)[None] / 2 + 0.25)])
    bits[0, 0] = synth.to_bf16_bits(np.array([127.0], np.float32))[0]         # scale 1: true halves among the quotients
    bits[0, 1:4] = synth.to_bf16_bits(np.array([0.5, 1.5, -2.5], np.float32))
    x = orc.bf16_to_f64(bits)
    q, s = orc.quantize_rows(x)
    assert q[0, 1:4].tolist() == [0, 2, -2]
    for r in range(x.shape[0]):
        most = Fraction(float(np.abs(x[r]).max()))
        assert Fraction(float(s[r])) == Fraction(float(np.float32(most / 127)))
        for j in range(x.shape[1]):
            assert q[r, j] == round(Fraction(float(x[r, j])) / Fraction(float(s[r])))   # round(): half to even


def test_gemm_and_experts_on_a_hand_example():
    X = np.zeros((1, 64), np.float32)
    X[0, :2] = 127.0, -2.0                                     # scale 1, codes 127 and -2
    bits = synth.to_bf16_bits(X)
    codes = np.zeros((2, 64), np.int8)
    codes[0, :2], codes[1, :2] = (3, 5), (-128, 1)
    np.testing.assert_array_equal(orc.i8_gemm(codes, [0.5, 2.0], bits), [[(381 - 10) * 0.5, (-128 * 127 - 2) * 2.0]])
    one = np.zeros((1, 64, 64), np.int8)
    one[0, 0, 0] = 1                                           # g = u = 127 * scale in column 0
    sc = np.full((1, 64), 1 / 127.0)
    y, slack, _ = orc.experts_i8((one, sc), (one, sc), (one, np.ones((1, 64))), bits, [[0, 7]], [[2.0, 5.0]])
    h = 1 / (1 + np.exp(-1.0))
    np.testing.assert_allclose(y[0, 0], 2.0 * h, rtol=1e-12)   # code 127 at scale h/127; id 7 names no expert
    assert not y[0, 1:].any() and (slack >= 0).all()
