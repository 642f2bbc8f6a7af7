"""Pins of oracle/layer.py: closed forms, brute force and central differences.
No GPU."""

import itertools

import numpy as np
import pytest

from oracle import layer as ol
from oracle import numerics as nu


def test_scores_closed_forms():
    x = np.array([[0.0, np.log(3.0), -np.inf], [np.nan, np.inf, 2.0], [-np.inf, np.nan, -np.inf]])
    assert np.allclose(ol.scores(x, False), [[0.25, 0.75, 0], [0, 1, 0], [0, 0, 0]])
    assert np.allclose(ol.scores(x, True), [[0.5, 0.75, 0], [0, 1, 1 / (1 + np.exp(-2))], [0, 0, 0]])


def test_choice_by_hand():
    x = np.array([[3.0, 3.0, 1.0, 2.0, 0.0, 5.0]])
    assert list(ol.gate(x, 3)[0][0]) == [5, 0, 1]                                     # a tie goes to the lower id
    assert list(ol.gate(x, 2, bias=np.array([0, 0, 2, 0, 0, 0.0]))[0][0]) == [2, 5]   # choices past the scores
    # groups {3, 3, 1} and {2, 0, 5}: by the largest the second, by the sums of the scores of two the first
    assert list(ol.gate(x, 2, n_groups=2, topk_groups=1)[0][0]) == [5, 3]
    y = np.array([[1.0, 1.0, -9.0, -9.0, -9.0, 1.5]])
    assert list(ol.gate(y, 2, sigmoid=True, n_groups=2, topk_groups=1, group_top=2)[0][0]) == [0, 1]
    idx, w = ol.gate(np.array([[1.0, -np.inf, np.nan, -np.inf]]), 2, renorm=True, scale=2.0)
    assert list(idx[0]) == [0, -1] and list(w[0]) == [2.0, 0.0]
    assert (ol.gate(x, 2, mask=[0])[0] == -1).all()


def test_renormed_weights_sum_to_one_far_out():
    for x in ([-200.0, -201.0], [300.0, 290.0], [-0.5, 0.5], [np.inf, 1.0]):
        for sigmoid in (False, True):
            w = ol.weights(np.array(x), None, sigmoid, True)
            assert np.isclose(w.sum(), 1)
    assert np.allclose(ol.weights(np.array([-200.0, -201.0]), None, True, True), [1 / (1 + np.exp(-1)), 1 / (1 + np.e)])


@pytest.mark.parametrize("sigmoid,renorm", itertools.product([False, True], repeat=2))
def test_gate_gradient_by_differences(sigmoid, renorm):
    rng = np.random.default_rng(1)
    x, idx = rng.standard_normal((3, 6)), np.array([[0, 4], [5, -1], [2, 3]])
    x[2, 0] = -np.inf
    g = rng.standard_normal((3, 2))

    def value(y):
        s, total = ol.scores(y, sigmoid), 0.0
        for t in range(3):
            live = [j for j in range(2) if idx[t, j] >= 0]
            w = ol.weights(y[t, idx[t, live]], s[t, idx[t, live]], sigmoid, renorm)
            total += 1.5 * (w * g[t, live]).sum()
        return total
    d, mag = ol.gate_bwd(x, idx, g, sigmoid, renorm, 1.5)
    for t in range(3):
        for e in range(6):
            if np.isfinite(x[t, e]):
                h = np.zeros_like(x)
                h[t, e] = 1e-5
                assert np.isclose(d[t, e], (value(x + h) - value(x - h)) / 2e-5, atol=1e-9)
    assert d[2, 0] == 0 and (np.abs(d) <= mag * (1 + 1e-12)).all()


def test_bias_update():
    b = ol.bias_update(np.array([1, 2, 3]), np.zeros(3, np.float32), 0.5)
    assert list(b) == [0.5, 0.0, -0.5]


def test_adamw_first_step_is_lr_times_sign():
    w, m, v, _, _ = ol.adamw(np.array([1.0, -2.0]), np.array([3.0, -1e-3]), np.zeros(2), np.zeros(2), 0.1, 0.9, 0.99, 0.0, 0.01, 1)
    assert np.allclose(w, [1 - 0.001 - 0.1, -2 + 0.002 + 0.1]) and np.allclose(m, [0.3, -1e-4]) and np.allclose(v, [0.09, 1e-8])


def test_random_bits_are_spread():
    r = ol.random16(7, 3, 1, 20000)
    assert abs(r.mean() / 65536 - 0.5) < 0.02 and len(np.unique(r)) > 16000
    assert not np.array_equal(r[:100], ol.random16(7, 4, 1, 100)) and not np.array_equal(r[:100], ol.random16(7, 3, 2, 100))


def test_int8_rows_and_product():
    rng = np.random.default_rng(2)
    x = nu.round_bf16(rng.standard_normal((4, 48)))
    x[2] = 0
    x[3, 5] = np.inf
    q, s = ol.quantize_int8(x)
    assert (np.abs(q[:2].astype(int)).max(1) == 127).all()
    assert (np.abs(q[:2] * s[:2, None] - x[:2]) <= 0.5001 * s[:2, None]).all()
    assert not q[2:].any() and s[2] == np.float32(2.0 ** -100) / np.float32(127) and np.isnan(s[3])
    b = rng.integers(-127, 128, (1, 3, 48)).astype(np.int8)
    bs = rng.random((1, 3)).astype(np.float32)
    c = ol.product_int8(q, s, b, bs, [2], [0], 4)
    assert np.isnan(c[2:]).all()
    assert np.isclose(c[1, 2], sum(int(q[1, i]) * int(b[0, 2, i]) for i in range(48)) * float(s[1]) * float(bs[0, 2]), rtol=1e-6)
