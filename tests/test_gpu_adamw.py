"""AdamW over lists of tensors (moe_adamw) against the float64 oracle.

Tolerances, every fp32 step off by half a step (2^-24 relative), square roots
and reciprocals of the hardware by a whole one: m and v are two products and a
sum of rounded constants and a scaled gradient, 6 roundings of the magnitudes
that make them.  The update lr m / den takes m's error and 10 roundings of its
own; the decayed weight 2, a bf16 weight one more (2^-8).  8-bit states: their
values are within half a step (to nearest) or one step (stochastic) of the
exact state on the grid of the block's scale."""

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
F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
U = 2.0 ** -24
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8)


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _at(n, dtype, off=0):
    """n elements, `off` elements behind a 16-byte boundary."""
    return torch.empty(n + off, dtype=dtype, device=DEV)[off:]


def _state(sizes, fp8=False, ptype=BF, gtype=None, master=False, seed=0, off=0, first=False):
    """A list's tensors; ptype None: both in turn."""
    g = torch.Generator(DEV).manual_seed(seed)
    s = dict(params=[], grads=[], m=[], v=[], master=[], m_scale=[], v_scale=[])
    for i, n in enumerate(sizes):
        pt = ptype or (BF, F32)[i % 2]
        rnd = lambda: torch.randn(n, generator=g, device=DEV)   # noqa: E731
        w = rnd()
        p, gr = _at(n, pt, off).copy_(w), _at(n, gtype or pt, off).copy_(rnd() * 0.1)
        s["params"].append(p)
        s["grads"].append(gr)
        s["master"].append(_at(n, F32, off).copy_(w) if master and pt == BF else None)
        m, v = rnd() * 0.02, (rnd() * 0.1).square()
        if first:
            m.zero_()
            v.zero_()
        if fp8:
            for name, x in (("m", m), ("v", v.sqrt())):
                sc = torch.from_numpy(ol.block_scale(x.double().cpu().numpy())).float().to(DEV)
                s[name].append(_at(n, F8, off).copy_((x / sc.repeat_interleave(128)[:n]).to(F8)))
                s[name + "_scale"].append(sc)
        else:
            s["m"].append(_at(n, F32, off).copy_(m))
            s["v"].append(_at(n, F32, off).copy_(v))
    if not fp8:
        s["m_scale"] = s["v_scale"] = None
    if not master:
        s["master"] = None
    return s


def _np(t):
    return t.double().cpu().numpy()


def _copy(s):
    return {k: None if v is None else [None if t is None else t.clone() for t in v] for k, v in s.items()}


def _check(s, step=7, wd=0.1, f=1.0, stochastic=False, seed=0, call=None, **kw):
    """One step of a list against the oracle, in place."""
    before, n_list = _copy(s), len(s["params"])
    decay = wd if isinstance(wd, list) else [wd] * n_list
    h = {**HYPER, **kw}
    mg.moe_adamw(**s, **h, step=step, weight_decay=wd, stochastic=stochastic, seed=seed, **(call or {}))
    for i in range(n_list):
        n = before["params"][i].numel()
        own = before["params"] if not before["master"] or before["master"][i] is None else before["master"]
        w, g, m, v = (_np(x[i]) for x in (own, before["grads"], before["m"], before["v"]))
        if s["m_scale"]:
            m = m * ol.spread(_np(before["m_scale"][i]), n)
            v = (v * ol.spread(_np(before["v_scale"][i]), n)) ** 2
        w1, m1, v1, mag, den = ol.adamw(w, g, m, v, h["lr"], h["beta1"], h["beta2"], h["eps"], decay[i], step, f)
        c1 = 1 - h["beta1"] ** step
        dm = 6 * U * mag
        upd = h["lr"] / c1 / den
        tol = upd * dm + 20 * U * upd * np.abs(m1) + 3 * U * np.abs(w) + 2.0 ** -149
        pt = before["params"][i].dtype
        final = tol + (2.0 ** -8 * (np.abs(w1) + tol) if pt == BF else 0)
        assert (np.abs(_np(s["params"][i]) - w1) <= final).all(), (i, n)
        if own is before["master"]:
            assert (np.abs(_np(s["master"][i]) - w1) <= tol).all()
            assert torch.equal(s["params"][i], s["master"][i].to(BF))
        dv = 8 * U * v1 + 2.0 ** -148
        if not s["m_scale"]:
            assert (np.abs(_np(s["m"][i]) - m1) <= dm + 2.0 ** -148).all()
            assert (np.abs(_np(s["v"][i]) - v1) <= dv).all()
            continue
        r1 = np.sqrt(v1)
        for name, x, dx in (("m", m1, dm), ("v", r1, 8 * U * r1 + 2.0 ** -74)):
            sc = _np(s[name + "_scale"][i])
            want = ol.block_scale(x)
            worst = np.zeros(len(sc) * 128)
            worst[:n] = dx
            assert (np.abs(sc - want) <= 4 * U * want + worst.reshape(-1, 128).max(1) / 448).all(), name
            scale = ol.spread(sc, n)
            code, y = _np(s[name][i]), x / scale
            slack = dx / scale + 6 * U * np.abs(y)
            if name == "m" or not stochastic:
                half = ol.e4m3_step(np.abs(y) + slack) / 2
                ok = np.abs(code - y) <= half * 1.0001 + slack
                ok |= (name == "v") & (y > 0) & (y <= 2.0 ** -10 + slack) & (code == 2.0 ** -9)
                assert ok.all(), name
            else:   # rounded up with the bits' probability; either way where they decide within the slack
                bits = ol.random16(seed, step, i, n) / 65536
                lo, hi = (_rounded(np.maximum(y + d, 0), bits) for d in (-slack, slack))
                assert ((code >= lo) & (code <= hi)).all()
        positive = r1 > 2.0 ** -60
        assert (_np(s["v"][i])[positive] > 0).all()
    for a, b in zip(s["grads"], before["grads"]):
        assert torch.equal(a, b)


def _rounded(y, bits):
    z = y + np.where(y < 2.0 ** -6, 2.0 ** -6, 0)
    step = ol.e4m3_step(z)
    q = np.floor(z / step + bits) * step - np.where(y < 2.0 ** -6, 2.0 ** -6, 0)
    return np.where((y > 0) & (q <= 0), 2.0 ** -9, np.minimum(q, 448.0))


SIZES = {
    "one_value": [1],
    "small_odd": [1, 7, 8, 9, 127, 128, 129, 255, 1000, 3],
    "pass_and_chunk_edges": [2047, 2048, 2049, 16383, 16384, 16385, 32768, 49153],
    "with_empty": [0, 5, 0, 4097, 0],
    "all_empty": [0, 0],
    "none": [],
    "more_than_one_launch": [3 + 37 * i % 400 for i in range(130)],
}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("fp8", [False, True])
def test_lists(name, fp8):
    _check(_state(SIZES[name], fp8, ptype=None, gtype=None if fp8 else F32))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ptype,master", [(BF, False), (BF, True), (F32, False), (None, True)])
@pytest.mark.parametrize("gtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_types_and_alignment(fp8, ptype, master, gtype, off):
    s = _state([5000, 260], fp8, ptype, gtype, master, seed=off, off=off)
    _check(s, wd=[0.0, 0.3])
    _check(s, step=8, wd=[0.0, 0.3])   # from the states that it left


def test_large():
    for fp8 in (False, True):
        _check(_state([5_000_003], fp8, seed=1, off=0), stochastic=False)


@pytest.mark.parametrize("fp8", [False, True])
def test_hyperparameters(fp8):
    for kw in (dict(beta1=0.0), dict(beta2=0.999, step=1), dict(beta2=0.0, eps=1.0), dict(lr=0.0), dict(eps=1e-3, step=100000), dict(lr=1.0, wd=-0.1)):
        _check(_state([777], fp8, F32, first=kw.get("step") == 1), **kw)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
def test_clipping(fp8, max_norm):
    s = _state([3000, 500], fp8, F32, master=False)
    total = torch.empty(1, dtype=torch.float64, device=DEV)
    mg.moe_grad_sumsq(tensors=s["grads"], sumsq=total, workspace=torch.empty(mg.moe_grad_workspace_size(2), dtype=torch.uint8, device=DEV))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    _check(s, f=ol.clip_factor(total.item(), max_norm), call=dict(sumsq=total, max_norm=max_norm, err_flag=err))
    assert err.item() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_no_step_without_a_norm(fp8, value):
    s = _state([3000, 500], fp8, master=True)
    before = _copy(s)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    mg.moe_adamw(**s, lr=0.1, sumsq=torch.full((1,), value, dtype=torch.float64, device=DEV), max_norm=1.0, err_flag=err)
    assert err.item() == mg.DEVERR_NONFINITE
    for k in s:
        for a, b in zip(s[k] or [], before[k] or []):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_values_that_are_not_finite():
    """A NaN stays with its element, an infinity with its block."""
    s = _state([400], True, F32)
    s["grads"][0][5] = float("nan")
    s["grads"][0][200] = float("inf")
    mg.moe_adamw(**s, **HYPER, stochastic=True, seed=3)
    m = (_np(s["m"][0]) * ol.spread(_np(s["m_scale"][0]), 400), _np(s["v"][0]) * ol.spread(_np(s["v_scale"][0]), 400))
    for x in m:
        assert np.isnan(x[5]) and np.isfinite(np.delete(x[:128], 5)).all() and np.isnan(x[128:256]).all() and np.isfinite(x[256:]).all()
    w = _np(s["params"][0])
    assert np.isnan(w[5]) and np.isfinite(np.delete(w, [5, 200])).all()
    t = _state([400], False, F32)
    t["grads"][0][5] = float("nan")
    mg.moe_adamw(**t, **HYPER)
    for x in (t["params"], t["m"], t["v"]):
        assert torch.isnan(x[0][5]) and torch.isfinite(x[0]).sum() == 399


@pytest.mark.parametrize("ptype", [BF, F32])
def test_stochastic_rounding(ptype):
    for seed, step in ((0, 1), (2 ** 32 - 1, 9), (12345, 2 ** 31 - 1)):
        _check(_state([1000, 129, 5], True, ptype, seed=2), step=step, stochastic=True, seed=seed)


def test_second_moment_follows_small_changes():
    """beta2 = 0.99 moves the root by less than a twelfth of a step: to nearest
    it stays, stochastically it follows in the mean.  4096 elements with one
    gradient each step and a few large ones that hold the blocks' scales."""
    n, steps = 4096, 300
    r0 = np.where(np.arange(n) % 128 == 0, 100.0, 10.0)
    g = torch.full((n,), 5.0, device=DEV)
    g[::128] = 100.0
    got = {}
    for stochastic in (False, True):
        sc = torch.from_numpy(ol.block_scale(r0)).float().to(DEV)
        s = dict(params=[torch.zeros(n, device=DEV)], grads=[g], m=[torch.zeros(n, device=DEV).to(F8)], v=[(torch.from_numpy(r0).to(DEV).float() / sc.repeat_interleave(128)).to(F8)],
                 m_scale=[torch.zeros(n // 128, device=DEV)], v_scale=[sc])
        for t in range(steps):
            mg.moe_adamw(**s, lr=0.0, beta2=0.99, step=t + 1, stochastic=stochastic, seed=1)
        got[stochastic] = np.delete(_np(s["v"][0]) * ol.spread(_np(s["v_scale"][0]), n), np.arange(0, n, 128)).mean()
    start = (10 / (100 / 448.0))
    want = np.sqrt(0.99 ** steps * 100 + (1 - 0.99 ** steps) * 25)   # 5.37
    assert abs(got[False] - 10) < 0.5 and start > 0
    # the root of the mean square is above the mean root: rounding noise of a
    # 2^-3 step has a variance of at most (step / 2)^2 each time, a part of the value of
    # 2^-4 squared, kept for 1 / (1 - beta2) steps times the step's small share
    assert abs(got[True] - want) < 0.15 * want


def test_repeats_bit_for_bit_and_in_any_split():
    """The same call gives the same bits; a list gives what its tensors give."""
    s = _state([70000, 300, 16384], True, master=True, seed=4)
    one, two, apart = _copy(s), _copy(s), _copy(s)
    kw = dict(**HYPER, step=3, weight_decay=0.1)
    mg.moe_adamw(**one, **kw)
    mg.moe_adamw(**two, **kw)
    for i in range(3):
        mg.moe_adamw(**{k: [v[i]] for k, v in apart.items()}, **kw)
    for k in s:
        for a, b, c in zip(one[k], two[k], apart[k]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(a.view(torch.uint8), c.view(torch.uint8))


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_steps_count_on(fp8):
    """Replays with the step and the rate on the device, against eager calls."""
    s = _state([5000, 77], fp8, master=True)
    mine = _copy(s)
    step, lr = torch.zeros(1, dtype=torch.int32, device=DEV), torch.full((1,), 1e-2, device=DEV)
    kw = dict(weight_decay=0.1, beta2=0.95, stochastic=fp8, seed=5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        mg.moe_adamw(**s, lr=0.0, step=0, step_dev=step, lr_dev=lr, **kw)
    side = torch.cuda.Stream()
    for t in range(1, 6):
        lr.fill_(1e-2 / t)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        mg.moe_adamw(**mine, lr=float(np.float32(1e-2 / t)), step=t, stream=side, **kw)
        torch.cuda.synchronize()
        for k in s:
            for a, b in zip(s[k] or [], mine[k] or []):
                # (the constants are made in fp64 on both sides and rounded once)
                if a.dtype in (F8,):
                    assert (a.view(torch.uint8) != b.view(torch.uint8)).float().mean() < 1e-3
                else:
                    assert torch.allclose(a.double(), b.double(), rtol=2.0 ** -7 if a.dtype == BF else 1e-5, atol=1e-6)


def test_rows_behind_the_last_element_stay():
    s = _state([1001], True, off=0)
    wide = {k: torch.full((1200,), 77, dtype=torch.uint8, device=DEV) for k in ("m", "v")}
    for k in wide:
        wide[k][:1001] = s[k][0].view(torch.uint8)
        s[k] = [wide[k][:1001]]
    scales = {k: torch.full((20,), 3.0, device=DEV) for k in ("m_scale", "v_scale")}
    for k in scales:
        scales[k][:8] = s[k][0]
        s[k] = [scales[k][:8]]
    mg.moe_adamw(**s, **HYPER)
    assert all((w[1001:] == 77).all() for w in wide.values()) and all((w[8:] == 3.0).all() for w in scales.values())


def test_refusals():
    s = _state([100, 50], False, master=True)
    e = _state([100, 50], True)
    for bad in (dict(grads=s["grads"][:1]), dict(m=s["m"] + s["m"]), dict(v=[s["v"][0].half(), s["v"][1]]), dict(m_scale=e["m_scale"]),
                dict(master=[s["m"][0], s["m"][0]]), dict(weight_decay=[0.1]), dict(weight_decay="x"), dict(params=s["params"][0]),
                dict(params=[t.double() for t in s["params"]]), dict(grads=[t.cpu() for t in s["grads"]]), dict(params=[s["params"][0], None]),
                dict(m=[s["m"][0][::2], s["m"][1]]), dict(sumsq=s["m"][0]), dict(step_dev=s["m"][0]), dict(lr_dev=torch.zeros(1, device=DEV).double())):
        with pytest.raises((ValueError, TypeError)):
            mg.moe_adamw(**{**s, "lr": 0.1, **bad})
    for bad in (dict(m_scale=[t[:0] for t in e["m_scale"]]), dict(v_scale=None), dict(m=s["m"])):
        with pytest.raises(ValueError):
            mg.moe_adamw(**{**e, "lr": 0.1, **bad})
    f = _state([100], False, F32)
    with pytest.raises(ValueError):
        mg.moe_adamw(**{**f, "master": [f["m"][0].clone()]}, lr=0.1)
    for bad in (dict(step=0), dict(beta1=1.0), dict(eps=-1.0), dict(lr=float("nan")), dict(v=f["m"])):
        with pytest.raises(mg.MoeError):
            mg.moe_adamw(**{**f, "lr": 0.1, **bad})
    with pytest.raises(OverflowError):
        mg.moe_adamw(**f, lr=0.1, seed=-1)


@pytest.mark.parametrize("n", [0, -3])
def test_a_step_below_one_counts_as_one(n):
    s = _state([3000], False, master=True)
    two = _copy(s)
    for t, at in ((s, n), (two, 1)):
        mg.moe_adamw(**t, lr=0.01, step_dev=torch.full((1,), at, dtype=torch.int32, device=DEV))
    for k in s:
        for a, b in zip(s[k] or [], two[k] or []):
            assert torch.equal(a, b) and torch.isfinite(a.float()).all()
