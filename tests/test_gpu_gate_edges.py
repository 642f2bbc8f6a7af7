"""The router's choice by scores (moe_router_gate) where equal and nearly equal
values decide, and in all of its plans for many tokens, against the float64 oracle.
Picks are compared exactly; the weights' tolerance is that of test_gpu_gate."""

import gc

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import layer as ol

from .test_gpu_gate import DEV, INF, _gate, _logits, _np

pytestmark = pytest.mark.gpu
MANY = 1500   # tokens: more than four a CU, so that tokens share a wave where their experts allow it


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """Tests after these measure what torch's allocator holds."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _check(x, k, sigmoid=False, bias=None, mask=None, rows=40, **kw):
    """One call against the oracle on a sample of the rows (the first and last among them); all
    rows' counts against the picks."""
    T, E = x.shape
    counts = torch.zeros(E, dtype=torch.int32, device=DEV)
    idx, probs = _gate(x, k, sigmoid, bias=bias, token_mask=mask, counts=counts, **kw)
    at = np.unique(np.r_[np.arange(min(T, 8)), T - 1, np.random.default_rng(T + E).integers(0, T, rows)]) if T > rows else np.arange(T)
    xn = _np(x[torch.from_numpy(at).to(DEV)])
    ref, w = ol.gate(xn, k, sigmoid, _np(bias), mask=None if mask is None else mask.cpu().numpy()[at], **kw)
    got = idx.cpu().numpy()
    bad = np.flatnonzero((got[at] != ref).any(1))
    assert not len(bad), (at[bad[:5]], got[at][bad[:5]], ref[bad[:5]])
    fin = np.where(np.isfinite(xn), xn, 0)
    d = np.abs(fin).max(1, keepdims=True) * 2 if not sigmoid or kw.get("renorm") else 0
    assert (np.abs(_np(probs)[at] - w) <= (d + 40) * 2.0 ** -23 * np.abs(w) + 2.0 ** -140).all()
    assert np.array_equal(counts.cpu().numpy(), np.bincount(got[got >= 0], minlength=E))
    return got


def _of(values, T, E, seed, dtype=torch.float32):
    g = torch.Generator(DEV).manual_seed(seed)
    v = torch.tensor(values, device=DEV, dtype=torch.float32)
    return v[torch.randint(0, len(values), (T, E), generator=g, device=DEV)].to(dtype)


SIZES = [(20, 4, 1), (20, 30, 5), (20, 64, 8), (20, 128, 8), (20, 256, 8), (20, 300, 6), (20, 512, 8), (20, 1024, 16),
         (MANY, 30, 5), (MANY, 64, 8), (MANY, 100, 4), (MANY, 128, 8), (MANY, 160, 8), (MANY, 256, 8), (MANY, 1024, 16)]


@pytest.mark.parametrize("T,E,groups", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_of_both_signs(T, E, groups, dtype):
    """-0 and +0 are equal: the lower id goes first."""
    k = min(E, 6)
    for values in ([-0.0, 0.0], [-0.0, 0.0, -0.0, 0.0, 1.0, -1.0], [-0.0, 0.0, -2.5, -INF]):
        x = _of(values, T, E, E + len(values), dtype)
        for sigmoid in (False, True):
            _check(x, k, sigmoid)
            if groups > 1:
                kw = dict(n_groups=groups, topk_groups=max(2, groups // 2), renorm=True)
                _check(x, min(k, E // groups * kw["topk_groups"]), sigmoid, **kw)


@pytest.mark.parametrize("T,E,groups", [s for s in SIZES if s[2] > 1])
@pytest.mark.parametrize("stay", [1, 2, 3])
def test_groups_go_by_logits_where_scores_are_equal(T, E, groups, stay):
    """Without a bias and judged by its largest choice, a group is judged by a logit:
    sigmoids of 40 and 60 are the same number, and so are softmax terms that underflow.
    Logits that are listed twice leave the order of picks open in fp32."""
    k = min(6, E // groups * stay)
    kw = dict(n_groups=groups, topk_groups=stay, group_top=1)
    near = [v + d for v in (25.3, 33.7, 38.51, 41.3, 47.9, 59.7) for d in (0.0, 4e-6, 8e-6)]
    for sigmoid, values in ((True, near), (True, near + [-INF] * 40 + [3.1] * 40), (False, near), (False, [100.7, -900.3, -1801.1, -900.30005, -2700.9]),
                            (False, [-900.3] * 3 + [-1801.1] * 30 + [0.7])):
        _check(_of(values, T, E, E + stay + len(values)), k, sigmoid, **kw)
    x = _logits(T, E, 3, spread=1.0)
    x[:, 1], x[:, -2:] = 38.5, 41.3
    _check(x, k, True, **kw)


PLANS = [(MANY, 30, 5), (MANY, 64, 8), (MANY, 100, 4), (MANY, 128, 8), (MANY, 160, 8), (MANY, 256, 8), (MANY, 260, 13), (MANY, 512, 8), (MANY, 1000, 8),
         (MANY, 1024, 32), (300, 300, 1), (300, 1024, 16), (9001, 30, 5), (9001, 64, 8), (9001, 100, 4), (9001, 256, 8)]   # (and larger workgroups)


@pytest.mark.parametrize("T,E,groups", PLANS)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens(T, E, groups, sigmoid, dtype):
    x = _logits(T, E, E, dtype)
    bias = 0.2 * torch.randn(E, generator=torch.Generator(DEV).manual_seed(E), device=DEV)
    _check(x, 8, sigmoid)
    _check(x, 4, sigmoid, renorm=True, scale=2.5)
    _check(x, 8, sigmoid, bias=bias, renorm=True)
    _check(x, 1, sigmoid, bias=bias)
    if groups == 1:
        return
    for top in (1, 2):
        for stay in (1, groups // 2):
            k = min(8, E // groups * stay)
            kw = dict(n_groups=groups, topk_groups=stay, group_top=top)
            _check(x, k, sigmoid, **kw, renorm=True)
            _check(x, k, sigmoid, bias=bias, **kw)


@pytest.mark.parametrize("T,E,groups", PLANS)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_many_tokens_masked_and_ruled_out(T, E, groups, sigmoid):
    g = torch.Generator(DEV).manual_seed(3)
    x = _logits(T, E, 3)
    x[torch.rand(T, E, generator=g, device=DEV) < 0.6] = -INF
    x[torch.rand(T, E, generator=g, device=DEV) < 0.1] = float("nan")
    x[1], x[2], x[3], x[5] = -INF, float("nan"), -INF, -INF
    x[3, E - 1] = 0.5
    x[4] = torch.finfo(torch.float32).min
    x[5, ::3] = torch.finfo(torch.float32).min
    mask = torch.rand(T, generator=g, device=DEV) < 0.8
    mask[3:6] = True
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    bias[E // 2], bias[E // 3] = -INF, float("nan")
    k = min(8, E // groups * max(1, groups // 2))
    for b in (None, bias):
        for kw in (dict(), dict(n_groups=groups, topk_groups=max(1, groups // 2), group_top=1 + (E % 3 != 0), renorm=True)):
            got = _check(x, k, sigmoid, bias=b, mask=mask, **kw)
            assert (got[1:3] == -1).all() and (got[~mask.cpu().numpy()] == -1).all()


@pytest.mark.parametrize("T,E,groups", PLANS + [(20, 64, 8), (20, 256, 8), (20, 1024, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_choices(T, E, groups, dtype):
    """Ties of single choices and of groups' sums, which are sums of the same two scores."""
    few = _of([0.0, 1.0, 2.0], T, E, 1).to(dtype)
    for sigmoid in (False, True):
        for x in (few, few - 90.0, few + 30.0):
            for bias in (None, torch.zeros(E, device=DEV), 0.25 * (torch.arange(E, device=DEV) % 3)):
                _check(x, 6, sigmoid, bias=bias)
                for top in (1, 2) if groups > 1 else ():
                    _check(x, min(6, E // groups * 2), sigmoid, bias=bias, n_groups=groups, topk_groups=2, group_top=top)
    # neighbours in fp32, in descending and ascending order of ids
    base = np.float32(1.5) + np.arange(E, dtype=np.float32) * np.float32(2.0 ** -23)
    for order in (base, base[::-1].copy()):
        x = torch.from_numpy(np.tile(order, (T, 1))).to(DEV)
        for kw in (dict(), dict(n_groups=groups, topk_groups=max(1, groups // 2))):
            k = min(6, E // groups * max(1, groups // 2))
            _check(x, k, rows=4, **kw)
            _check(x, k, True, bias=torch.full((E,), 3.0, device=DEV), rows=4, **kw)


@pytest.mark.parametrize("T,E,groups", PLANS)
@pytest.mark.parametrize("spread", [1e-6, 1e-3, 30.0, 1e4])
def test_narrow_and_wide_logits(T, E, groups, spread):
    """Far out, scores are 0 and 1 and sums of them and a bias decide: all in 64 bits."""
    x = _logits(T, E, 7, spread=spread)
    bias = 1e-3 * torch.randn(E, generator=torch.Generator(DEV).manual_seed(4), device=DEV)
    stay = max(1, groups // 2)
    k = min(8, E // groups * stay)
    for sigmoid in (False, True):
        _check(x, k, sigmoid, renorm=True)
        for top in (1, 2):
            kw = dict(n_groups=groups, topk_groups=stay, group_top=top)
            _check(x, k, sigmoid, bias=bias, **kw)
            _check(x - 300.0, k, sigmoid, bias=bias, renorm=True, **kw)
            _check(x, k, sigmoid, renorm=True, **kw)


@pytest.mark.parametrize("T,E,groups", [(9, 16, 1), (9, 64, 8), (9, 256, 8), (MANY, 64, 8), (MANY, 256, 8), (MANY, 1024, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_picks_of_infinite_logits(T, E, groups, dtype):
    x = _logits(T, E, 1, dtype)
    x[0, 3] = INF
    x[1, 5] = x[1, 9] = INF
    x[2, 0] = 1e30
    x[3, -3:] = INF
    x[4] = INF
    x[5, ::2], x[5, 1::2] = INF, -INF
    bias = 0.1 * torch.randn(E, generator=torch.Generator(DEV).manual_seed(4), device=DEV)
    bias[E - 5] = INF
    for sigmoid in (False, True):
        for b in (None, bias):
            for renorm in (False, True):
                _check(x, 4, sigmoid, bias=b, renorm=renorm, rows=9)
                if groups > 1:
                    for top in (1, 2):
                        _check(x, 4, sigmoid, bias=b, renorm=renorm, rows=9, n_groups=groups, topk_groups=2, group_top=top)


@pytest.mark.parametrize("T,E", [(8, 16), (8, 128), (8, 300), (MANY, 64), (MANY, 256)])
def test_weights_and_gradients_of_tiny_sigmoids(T, E):
    """Renormalised weights of scores that are subnormal numbers beside a small sum: as
    exact as others, while the weight itself is a normal number (2^-126)."""
    k = 4
    x = torch.full((T, E), -200.0, device=DEV)
    rows = [(-11.7, -101.66, -48.0, -97.3), (-60.0, -100.0, -103.2, -90.0), (-68.9, -103.9, -110.0, -150.0), (3.0, -84.2, -87.5, -1.0),
            (-103.0, -103.5, -110.0, -120.0), (-69.1, -69.0, -104.5, -87.4), (80.0, -6.0, 30.0, 0.5), (-40.0, -126.0, -122.0, -43.0)]
    g = torch.Generator(DEV).manual_seed(1)
    for t in range(T):
        at = torch.randperm(E, generator=g, device=DEV)[:k]
        x[t, at] = torch.tensor(rows[t % len(rows)], device=DEV)
    got = _check(x, k, True, renorm=True, rows=16)
    idx = torch.from_numpy(got).to(DEV).int()
    d = torch.randn(T, k, generator=g, device=DEV)
    out = torch.empty_like(x)
    mg.moe_router_gate_bwd(T=T, E=E, k=k, logits=x, expert_idx=idx, dprobs=d, dlogits=out, score=mg.SCORE_SIGMOID, renorm=True)
    n = 40
    ref, mag = ol.gate_bwd(_np(x[:n]), got[:n], _np(d[:n]), True, renorm=True)
    assert (np.abs(_np(out[:n]) - ref) <= (400 + 40) * 2.0 ** -23 * mag + 2.0 ** -140).all()
