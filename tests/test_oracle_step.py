"""Pins of the oracle of the block-scaled FP8 products, the router's losses
and the gradient norm (oracle/step.py): closed forms, brute force and central
differences.  No GPU."""

import numpy as np
import pytest

from oracle import numerics as nu
from oracle import step as st


def test_block_scales_closed_forms():
    s, r = st.block_scales(np.array([448.0, 896.0, 1.0, 0.0]))
    assert s[0] == 1 and r[0] == 1 and s[1] == 2 and r[1] == 0.5
    assert s[2] == np.float32(1) / np.float32(448) and r[2] == 448
    assert s[3] == np.float32(2.0 ** -100) / np.float32(448)
    s, r = st.block_scales(np.array([448.0, 449.0, 447.0, 7.0, 7.03125, 1e30]), pow2=True)
    assert list(s[:5]) == [1.0, 2.0, 1.0, 2.0 ** -6, 2.0 ** -5]
    assert np.all(s * r == 1)
    assert s[5] >= 1e30 / 448 > s[5] / 2


@pytest.mark.parametrize("pow2", [False, True])
def test_codes_are_nearest_and_in_range(pow2):
    rng = np.random.default_rng(0)
    x = nu.round_bf16(rng.standard_normal((5, 300)) * np.exp(3 * rng.standard_normal((5, 1))))
    q, s = st.quantize_rows(x, pow2)
    v = st.dequantize_rows(q, s)
    sc = np.repeat(s.T.astype(np.float64), 128, axis=1)[:, :300]
    assert np.all(np.abs(x) <= 448.0001 * sc)
    # half a step: 2^-4 relative, or half of 2^-9 scales near zero
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x) * 1.001, 2.0 ** -10 * sc * 1.001))


def test_tiles_agree_with_their_transpose_and_with_rows_on_one_value():
    rng = np.random.default_rng(1)
    x = nu.round_bf16(rng.standard_normal((200, 144)))
    q, s = st.quantize_tiles(x)
    qt, sT = st.quantize_tiles(x.T)
    assert np.array_equal(q.T, qt) and np.array_equal(s.T, sT)
    y = np.where(rng.random((128, 128)) < 0.5, -3.0, 3.0)   # every block's maximum is 3
    assert np.array_equal(st.quantize_tiles(y)[0], st.quantize_rows(y)[0])


def test_grouped_products_by_brute_force():
    rng = np.random.default_rng(2)
    a, w = rng.standard_normal((7, 5)), rng.standard_normal((2, 3, 5))
    c, mag = st.grouped_product(a, w, [2, 3], [0, 3])
    assert np.isnan(c[2]).all() and np.isnan(c[6]).all()
    for r, e in ((0, 0), (1, 0), (3, 1), (5, 1)):
        for n in range(3):
            assert np.isclose(c[r, n], sum(a[r, k] * w[e, n, k] for k in range(5)))
    aT, bT = rng.standard_normal((3, 384)), rng.standard_normal((2, 384))
    g, _ = st.grouped_weight_grad(aT, bT, [130, 0], [0, 256])
    assert np.allclose(g[0], sum(np.outer(aT[:, m], bT[:, m]) for m in range(256)))
    assert not g[1].any()


def _loss_of(x, idx, mask, balance, zc, dprobs, g, counts, n):
    """The scalar whose gradient router_bwd is, counts held fixed."""
    p, lse, any_ = st._softmax(x)
    keep = any_ & (np.ones(len(x), bool) if mask is None else mask)
    k, E = idx.shape[1], x.shape[1]
    L = g[0] * balance * E * (counts / (k * n) * p[keep].sum(0) / n).sum()
    L += g[1] * zc * (lse[keep] ** 2).sum() / n
    for s in range(k):
        L += (p[np.arange(len(x)), idx[:, s]] * dprobs[:, s]).sum()
    return L


@pytest.mark.parametrize("masked", [False, True])
def test_router_gradient_by_central_differences(masked):
    rng = np.random.default_rng(3)
    T, E, k = 6, 5, 2
    x = rng.standard_normal((T, E))
    idx = np.argsort(-x, axis=1)[:, :k].astype(np.int32)
    idx[1] = [2, 2]                       # one expert listed twice
    mask = np.array([1, 0, 1, 1, 0, 1], bool) if masked else None
    dprobs, g = rng.standard_normal((T, k)), (0.7, -1.3)
    counts, n, mean, loss = st.router_loss(x, idx, mask, 0.4, 0.2)
    assert counts.sum() == n * k and np.isclose(mean.sum(), 1)
    d, _ = st.router_bwd(x, idx, dprobs, g, counts, n, mask, 0.4, 0.2)
    for t in range(T):
        for e in range(E):
            h = 1e-5
            xp, xm = x.copy(), x.copy()
            xp[t, e] += h
            xm[t, e] -= h
            num = (_loss_of(xp, idx, mask, 0.4, 0.2, dprobs, g, counts, n)
                   - _loss_of(xm, idx, mask, 0.4, 0.2, dprobs, g, counts, n)) / (2 * h)
            assert abs(num - d[t, e]) < 1e-8


def test_router_loss_closed_forms():
    # uniform probabilities and even counts: balance_coef * 1; lse = log E
    T, E, k = 8, 4, 1
    x = np.zeros((T, E))
    idx = (np.arange(T) % E)[:, None].astype(np.int32)
    counts, n, mean, loss = st.router_loss(x, idx, None, 0.5, 2.0)
    assert np.isclose(loss[0], 0.5) and np.isclose(loss[1], 2.0 * np.log(4) ** 2)
    # nothing kept
    counts, n, mean, loss = st.router_loss(x, idx, np.zeros(T), 0.5, 2.0)
    assert n == 0 and not counts.any() and loss == (0.0, 0.0)
    # a row of -inf is left out; ids outside the range count nowhere
    x[0] = -np.inf
    idx[1] = -1
    counts, n, mean, loss = st.router_loss(x, idx, None, 0.5, 2.0)
    assert n == T - 1 and counts.sum() == T - 2
    d, _ = st.router_bwd(x, idx, np.ones((T, k)), None, counts, n, None, 0.5, 2.0)
    assert np.isfinite(d).all() and not d[0].any()


def test_clip_closed_forms():
    g = [np.array([3.0, 0.0]), np.array([4.0])]
    assert st.grad_norm(g) == 5.0
    assert np.isclose(st.clip_factor(5.0, 2.5), 0.5, rtol=1e-6)
    assert st.clip_factor(5.0, 10.0) == 1.0 and st.clip_factor(np.inf, 1.0) == 1.0
