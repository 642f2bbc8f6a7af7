"""The router's choice by scores (moe_router_gate), its gradient and the bias
update against the float64 oracle.

Picks are compared exactly.  Tolerances of the weights, from fp32 arithmetic
whose steps are each off by half a step (2^-24 relative) and exponentials by
one (2^-23): a difference to the largest logit, rounded, scales an exponential
by up to |d| 2^-24; then up to 1024 terms are added over 16 registers and 6
lane exchanges (22 roundings), divided and scaled.  In all (|d| + 40) 2^-23 of
the value, and 2^-140 where it leaves the normal range.  Gradients are sums of
such products: the same of the sum of their magnitudes; bf16 ones are rounded
once more (2^-8)."""

import gc

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import layer as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """Tests after these measure what torch's allocator holds."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


DEV = "cuda"
INF = float("inf")


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _logits(T, E, seed=0, dtype=torch.float32, spread=1.0):
    g = torch.Generator(DEV).manual_seed(seed)
    return (spread * (torch.randn(T, E, generator=g, device=DEV) + torch.randn(1, E, generator=g, device=DEV))).to(dtype)


def _gate(x, k, sigmoid=False, T=None, E=None, counts=None, **kw):
    T, E = T or x.shape[0], E or x.shape[1]
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    probs = torch.full((T, k), float("nan"), device=DEV)
    mg.moe_router_gate(T=T, E=E, k=k, logits=x, expert_idx=idx, probs=probs, counts=counts,
                       score=mg.SCORE_SIGMOID if sigmoid else mg.SCORE_SOFTMAX, **kw)
    return idx, probs


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _check(x, k, sigmoid=False, bias=None, mask=None, **kw):
    """One call against the oracle; returns its picks."""
    T, E = x.shape
    counts = torch.full((E,), 5, dtype=torch.int32, device=DEV)
    idx, probs = _gate(x, k, sigmoid, bias=bias, token_mask=mask, counts=counts, **kw)
    xn = _np(x)
    ref, w = ol.gate(xn, k, sigmoid, _np(bias), mask=None if mask is None else mask.cpu().numpy(), **kw)
    got = idx.cpu().numpy()
    bad = np.flatnonzero((got != ref).any(1))
    assert not len(bad), (bad[:5], got[bad[:5]], ref[bad[:5]])
    fin = np.where(np.isfinite(xn), xn, 0)
    d = np.abs(fin).max(1, keepdims=True) * 2 if not sigmoid or kw.get("renorm") else 0
    assert (np.abs(_np(probs) - w) <= (d + 40) * 2.0 ** -23 * np.abs(w) + 2.0 ** -140).all()
    assert np.array_equal(counts.cpu().numpy() - 5, np.bincount(ref[ref >= 0], minlength=E))
    return ref


SHAPES = [(1, 1, 1), (3, 2, 2), (7, 5, 3), (64, 8, 2), (65, 32, 8), (33, 33, 4), (50, 60, 6), (50, 64, 8), (40, 100, 7), (40, 128, 8),
          (37, 160, 6), (36, 256, 8), (9, 300, 8), (10, 512, 5), (6, 1000, 8), (5, 1024, 8)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_without_groups(T, E, k, sigmoid, dtype):
    x = _logits(T, E, T + E, dtype)
    bias = 0.2 * torch.randn(E, generator=torch.Generator(DEV).manual_seed(E), device=DEV)
    for kw in (dict(), dict(renorm=True, scale=2.5), dict(bias=bias), dict(bias=bias, renorm=True)):
        _check(x, k, sigmoid, **kw)


GROUPS = [(20, 256, 8, 8, 4), (20, 256, 8, 8, 1), (21, 160, 6, 8, 3), (10, 64, 4, 16, 5), (10, 128, 2, 64, 2), (7, 1024, 8, 32, 3),
          (7, 15, 3, 3, 2), (6, 35, 4, 5, 2), (5, 1020, 8, 5, 2), (5, 1017, 8, 9, 4), (5, 986, 8, 17, 3), (5, 1023, 8, 33, 6), (9, 24, 3, 24, 5),
          (4, 64, 8, 64, 40), (30, 8, 2, 4, 4)]


@pytest.mark.parametrize("T,E,k,groups,stay", GROUPS)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("top", [1, 2])
def test_groups(T, E, k, groups, stay, sigmoid, top):
    bias = 0.2 * torch.randn(E, generator=torch.Generator(DEV).manual_seed(E), device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        x = _logits(T, E, T + E, dtype)
        _check(x, k, sigmoid, n_groups=groups, topk_groups=stay, group_top=top, renorm=True)
        _check(x, k, sigmoid, bias=bias, n_groups=groups, topk_groups=stay, group_top=top)


@pytest.mark.parametrize("E,groups", [(8, 1), (64, 1), (256, 8), (512, 1)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_masks_and_ruled_out_experts(E, groups, sigmoid):
    T, k = 70, min(8, E)
    g = torch.Generator(DEV).manual_seed(3)
    x = _logits(T, E, 3)
    x[torch.rand(T, E, generator=g, device=DEV) < 0.6] = -INF
    x[torch.rand(T, E, generator=g, device=DEV) < 0.1] = float("nan")
    x[1], x[2], x[3] = -INF, float("nan"), -INF
    x[3, E - 1] = 0.5                        # one expert is left
    x[4] = torch.finfo(torch.float32).min    # all equal, and still experts
    x[5, :] = -INF
    x[5, ::3] = torch.finfo(torch.float32).min
    mask = torch.rand(T, generator=g, device=DEV) < 0.8
    mask[3:6] = True
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    bias[E // 2] = -INF
    bias[E // 3] = float("nan")
    kw = dict(n_groups=groups, topk_groups=max(1, groups // 2), group_top=2, renorm=True) if groups > 1 else {}
    for b in (None, bias):
        for m in (None, mask, mask.to(torch.uint8)):
            ref = _check(x, k, sigmoid, bias=b, mask=m, **kw)
            assert (ref[1] == -1).all() and (ref[2] == -1).all() and ref[3, 0] in (E - 1, -1)


def test_infinite_logits():
    x = _logits(4, 16, 1)
    x[0, 3] = INF
    x[1, 5] = x[1, 9] = INF
    x[2, 0] = 1e30
    for sigmoid in (False, True):
        for renorm in (False, True):
            _, w = _gate(x, 3, sigmoid, renorm=renorm)
            ref, v = ol.gate(_np(x), 3, sigmoid, renorm=renorm)
            assert np.allclose(_np(w), v, rtol=2e-5, atol=1e-30), (sigmoid, renorm)
            _, got = _gate(x, 3, sigmoid, renorm=renorm)
            assert torch.equal(w, got)


@pytest.mark.parametrize("E,groups", [(64, 1), (256, 1), (256, 8), (1024, 1), (30, 5)])
def test_equal_choices_go_to_the_lower_id(E, groups):
    """Ties of every kind, and choices that differ by less than fp32 shows."""
    k = 6
    kw = dict(n_groups=groups, topk_groups=2, group_top=2) if groups > 1 else {}
    zero = torch.zeros(3, E, device=DEV)
    few = torch.randint(0, 3, (50, E), generator=torch.Generator(DEV).manual_seed(1), device=DEV).float()
    for sigmoid in (False, True):
        for x in (zero, few, few - 90.0, few + 30.0):
            for bias in (None, torch.zeros(E, device=DEV), 0.25 * (torch.arange(E, device=DEV) % 3)):
                if groups > 1 and bias is None and not sigmoid:
                    continue   # sums of equal scores in another order: equal in numbers, not in the last bit
                _check(x, k, sigmoid, bias=bias, **kw)
    # neighbours in fp32, in descending and ascending order of ids
    base = np.float32(1.5) + np.arange(E, dtype=np.float32) * np.float32(2.0 ** -23)
    for order in (base, base[::-1].copy()):
        x = torch.from_numpy(np.tile(order, (4, 1))).to(DEV)
        _check(x, k)
        _check(x, k, True, bias=torch.zeros(E, device=DEV))
        _check(x, k, True, bias=torch.full((E,), 3.0, device=DEV))


@pytest.mark.parametrize("spread", [1e-6, 1e-3, 30.0, 1e4])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_narrow_and_wide_logits(spread, sigmoid):
    x = _logits(60, 256, 7, spread=spread)
    bias = 1e-3 * torch.randn(256, generator=torch.Generator(DEV).manual_seed(4), device=DEV)
    _check(x, 8, sigmoid, renorm=True)
    _check(x, 8, sigmoid, bias=bias)
    if spread < 1e4:   # (far out, sums of scores are equal numbers with other last bits)
        _check(x, 8, sigmoid, bias=bias, n_groups=8, topk_groups=4, group_top=2, renorm=True)
    _check(x - 300.0, 8, sigmoid, renorm=True)


def test_agrees_with_the_softmax_router():
    x = _logits(333, 128, 5)
    idx, probs = _gate(x, 8)
    i2, p2 = torch.empty_like(idx), torch.empty_like(probs)
    mg.moe_router_topk(T=333, E=128, k=8, logits=x, expert_idx=i2, probs=p2)
    assert torch.equal(idx, i2) and torch.allclose(probs, p2, rtol=1e-5, atol=0)


@pytest.mark.parametrize("E,ld", [(60, 61), (64, 72), (256, 260), (200, 203)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_apart_and_odd_addresses(E, ld, dtype):
    """Strides, and buffers aligned to their type alone."""
    T, k = 21, 5
    x = _logits(T, E, 2, dtype)
    want = _gate(x, k, True, renorm=True)
    flat = torch.full((T * ld + 1,), float("nan"), dtype=dtype, device=DEV)
    rows = flat[1:].view(T, ld)
    rows[:, :E] = x
    assert all(torch.equal(a, b) for a, b in zip(_gate(flat[1:], k, True, T=T, E=E, ld=ld, renorm=True), want))
    d = 0.1 * torch.randn(T, k, generator=torch.Generator(DEV).manual_seed(1), device=DEV)
    ref = _bwd(x, want[0], d, True, renorm=True)
    out = torch.full((T * ld + 1,), 3.0, dtype=dtype, device=DEV)
    mg.moe_router_gate_bwd(T=T, E=E, k=k, logits=flat[1:], expert_idx=want[0], dprobs=d, dlogits=out[1:], score=mg.SCORE_SIGMOID,
                           renorm=True, ld=ld, ld_d=ld)
    assert torch.equal(out[1:].view(T, ld)[:, :E], ref) and (out[1:].view(T, ld)[:, E:] == 3.0).all() and out[0] == 3.0


def test_no_tokens():
    e = torch.empty(0, 8, device=DEV)
    _gate(e, 2, T=0, E=8)
    mg.moe_router_gate_bwd(T=0, E=8, k=2, logits=e, expert_idx=torch.empty(0, 2, dtype=torch.int32, device=DEV),
                           dprobs=torch.empty(0, 2, device=DEV), dlogits=e)
    torch.cuda.synchronize()


def test_many_tokens():
    """More than one token a lane group and workgroup; a sample of rows."""
    x = _logits(20011, 256, 9)
    bias = 0.1 * torch.randn(256, generator=torch.Generator(DEV).manual_seed(2), device=DEV)
    kw = dict(bias=bias, n_groups=8, topk_groups=4, group_top=2, renorm=True)
    counts = torch.zeros(256, dtype=torch.int32, device=DEV)
    idx, probs = _gate(x, 8, True, counts=counts, **kw)
    at = torch.randperm(20011, generator=torch.Generator().manual_seed(1))[:400].to(DEV)
    ref, w = ol.gate(_np(x[at]), 8, True, **{**kw, "bias": _np(bias)})
    assert np.array_equal(idx[at].cpu().numpy(), ref) and np.allclose(_np(probs[at]), w, rtol=1e-5)
    assert torch.equal(counts.long(), torch.bincount(idx.flatten().long(), minlength=256))


# ---------------------------------------------------------------- gradient --
def _bwd(x, idx, d, sigmoid, out=None, **kw):
    out = torch.full_like(x, float("nan")) if out is None else out
    mg.moe_router_gate_bwd(T=x.shape[0], E=x.shape[1], k=idx.shape[1], logits=x, expert_idx=idx, dprobs=d, dlogits=out,
                           score=mg.SCORE_SIGMOID if sigmoid else mg.SCORE_SOFTMAX, **kw)
    return out


def _check_bwd(x, idx, d, sigmoid, before=None, **kw):
    got = _bwd(x, idx, d, sigmoid, out=None if before is None else before.clone(), accumulate=before is not None, **kw)
    xn = _np(x)
    ref, mag = ol.gate_bwd(xn, idx.cpu().numpy(), _np(d), sigmoid, **kw)
    spread = 2 * np.abs(np.where(np.isfinite(xn), xn, 0)).max(1, keepdims=True)
    tol = (spread + 40) * 2.0 ** -23 * mag + 2.0 ** -140
    if before is not None:
        ref = ref + _np(before)
        tol = tol + 2.0 ** -24 * np.abs(ref)
    if x.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    diff = np.abs(_np(got) - ref)
    assert (diff <= tol).all(), (diff - tol).max()


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient(T, E, k, sigmoid, dtype):
    x = _logits(T, E, T + E, dtype)
    idx, _ = _gate(x, k, sigmoid)
    g = torch.Generator(DEV).manual_seed(E)
    idx[torch.rand(T, k, generator=g, device=DEV) < 0.2] = -1
    d = torch.randn(T, k, generator=g, device=DEV)
    d[idx < 0] = float("nan")   # dropped slots have no part
    before = torch.randn(T, E, generator=g, device=DEV).to(dtype)
    for renorm in (False, True):
        _check_bwd(x, idx, d, sigmoid, renorm=renorm, scale=1.5)
        _check_bwd(x, idx, d, sigmoid, before=before, renorm=renorm)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_edges(sigmoid, renorm):
    T, E, k = 9, 40, 4
    x = _logits(T, E, 1)
    g = torch.Generator(DEV).manual_seed(1)
    idx = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    idx[0] = 7                                    # one expert four times
    idx[1] = torch.tensor([-1, E, 2 ** 31 - 1, 3], device=DEV, dtype=torch.int32)   # ids outside
    idx[2] = -1
    x[2] = float("nan")
    x[3, idx[3, 1].item()] = -INF                 # a pick that is ruled out since
    x[4] = -INF
    x[5] -= 200.0
    x[6] *= 30.0
    x[7, :30] = float("nan")
    idx[7] = torch.tensor([30, 31, 39, 35], device=DEV, dtype=torch.int32)
    d = torch.randn(T, k, generator=g, device=DEV)
    _check_bwd(x, idx, d, sigmoid, renorm=renorm)
    out = _bwd(x, idx, d, sigmoid, renorm=renorm)
    assert not out[2].any() and not out[4].any()
    y = x.clone()   # in place of the logits
    assert torch.equal(_bwd(y, idx, d, sigmoid, out=y, renorm=renorm), out)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradient_by_differences(sigmoid):
    """Of the weights that the forward call itself gives."""
    x = _logits(6, 24, 3)
    idx, _ = _gate(x, 4, sigmoid, renorm=True, scale=2.0)
    d = torch.randn(6, 4, generator=torch.Generator(DEV).manual_seed(1), device=DEV)
    got = _np(_bwd(x, idx, d, sigmoid, renorm=True, scale=2.0))
    h = 1e-2
    for t, e in ((0, idx[0, 1].item()), (3, idx[3, 0].item()), (5, idx[5, 2].item())):
        v = []
        for sign in (1, -1):
            y = x.clone()
            y[t, e] += sign * h
            i2, w = _gate(y, 4, sigmoid, renorm=True, scale=2.0)
            at = {int(i): float(p) for i, p in zip(i2[t], w[t])}
            if set(at) != set(idx[t].tolist()):
                break
            v.append(sum(at[int(i)] * float(p) for i, p in zip(idx[t], d[t])))
        if len(v) == 2:   # weights of about 1 off by 2^-22 over 2 h, and h^2 of the third derivative
            assert abs((v[0] - v[1]) / (2 * h) - got[t, e]) <= 4 * 8 * 2.0 ** -22 / (2 * h) + 8 * h * h


# ------------------------------------------------------------- bias, use ----
@pytest.mark.parametrize("E", [1, 7, 64, 256, 1024])
@pytest.mark.parametrize("reset", [False, True])
def test_bias_update(E, reset):
    g = torch.Generator(DEV).manual_seed(E)
    counts = torch.randint(0, 5, (E,), generator=g, device=DEV, dtype=torch.int32)
    if E > 1:
        counts[0] = 2 ** 31 - 1   # sums past 32 bits
    bias = torch.randn(E, generator=g, device=DEV)
    want = ol.bias_update(counts.cpu().numpy(), bias.cpu().numpy(), 1e-3)
    c = counts.clone()
    mg.moe_router_bias_update(E=E, counts=c, bias=bias, rate=1e-3, reset=reset)
    assert np.array_equal(bias.cpu().numpy(), want)
    assert torch.equal(c, torch.zeros_like(c) if reset else counts)


def test_captured_with_another_stream():
    """Replays with other inputs, eager calls between them on another stream."""
    T, E, k = 300, 64, 4
    x, bias = _logits(T, E, 0), torch.zeros(E, device=DEV)
    idx, probs = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    counts, d, dx = torch.zeros(E, dtype=torch.int32, device=DEV), torch.randn(T, k, device=DEV), torch.empty(T, E, device=DEV)

    def step(x, idx, probs, counts, bias, dx, stream=None):
        kw = dict(T=T, E=E, k=k, logits=x, expert_idx=idx, score=mg.SCORE_SIGMOID, renorm=True, stream=stream)
        mg.moe_router_gate(**kw, probs=probs, bias=bias, counts=counts)
        mg.moe_router_gate_bwd(**kw, dprobs=d, dlogits=dx)
        mg.moe_router_bias_update(E=E, counts=counts, bias=bias, rate=0.01, reset=True, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, idx, probs, counts, bias, dx)
    eager_bias = torch.zeros(E, device=DEV)
    for seed in range(4):
        y = _logits(T, E, seed)
        x.copy_(y)
        graph.replay()
        mine = [torch.empty_like(idx), torch.empty_like(probs), torch.zeros_like(counts), eager_bias, torch.empty_like(dx)]
        s.wait_stream(torch.cuda.current_stream())
        step(y, *mine, stream=s)
        torch.cuda.synchronize()
        for a, b in zip((idx, probs, counts, bias, dx), mine):
            assert torch.equal(a, b)


def test_refusals():
    x = torch.zeros(4, 8, device=DEV)
    idx, probs = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    ok = dict(T=4, E=8, k=2, logits=x, expert_idx=idx, probs=probs)
    for bad in (dict(logits=x.double()), dict(logits=x[:3]), dict(logits=x.t()), dict(logits=x.cpu()), dict(expert_idx=idx.long()),
                dict(probs=probs[:3]), dict(bias=x[0, :7]), dict(bias=x[0].double()), dict(token_mask=idx[:, 0]), dict(counts=probs),
                dict(ld=9), dict(T=5)):
        with pytest.raises(ValueError):
            mg.moe_router_gate(**{**ok, **bad})
    for bad in (dict(k=9), dict(scale=INF), dict(score=2), dict(n_groups=3, topk_groups=1), dict(n_groups=4, topk_groups=5)):
        with pytest.raises((mg.MoeError, ValueError)):
            mg.moe_router_gate(**{**ok, **bad})
    back = dict(T=4, E=8, k=2, logits=x, expert_idx=idx, dprobs=probs, dlogits=torch.empty_like(x))
    for bad in (dict(dlogits=x.bfloat16()), dict(logits=x.bfloat16()), dict(dprobs=probs.double()), dict(dlogits=x[:2]), dict(ld_d=10)):
        with pytest.raises(ValueError):
            mg.moe_router_gate_bwd(**{**back, **bad})
