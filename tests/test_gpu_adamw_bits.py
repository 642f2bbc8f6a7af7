"""AdamW with 8-bit states (moe_adamw), bit for bit.

The states' arithmetic is fixed: every product, sum, quotient and root of a state
is rounded to fp32 by itself, and so is the clipping factor, once, from fp64.  So
codes and scales are compared for equality with the same operations in NumPy."""

import gc

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import layer as ol

from .test_gpu_adamw import BF, DEV, F32, HYPER, _copy, _rounded, _state

pytestmark = pytest.mark.gpu
f4 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """Tests after these measure what torch's allocator holds."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _f32(t):
    return t.float().cpu().numpy()


def _blocks(x):
    p = np.zeros(-(-len(x) // 128) * 128, dtype=f4)
    p[:len(x)] = np.abs(x)
    return np.maximum(p.reshape(-1, 128).max(1), f4(2.0 ** -100))


def _spread(s, n):
    return np.repeat(s, 128)[:n]


def _nearest(y):
    return torch.from_numpy(y).to(torch.float8_e4m3fn).float().numpy()


def expected(s, i, f=1.0, step=7, stochastic=False, seed=0, beta1=0.9, beta2=0.95, **_):
    """Codes' values and scales of tensor i after a step: (m, m_scale, (least, largest) of v, v_scale)."""
    n, f = s["grads"][i].numel(), f4(f)
    d = _f32(s["grads"][i]) * f
    m = _f32(s["m"][i]) * _spread(_f32(s["m_scale"][i]), n)
    r = _f32(s["v"][i]) * _spread(_f32(s["v_scale"][i]), n)
    m = f4(beta1) * m + f4(1 - beta1) * d
    r = np.sqrt(f4(beta2) * (r * r) + f4(1 - beta2) * d * d)
    mm, rr = _blocks(m), _blocks(r)
    y = r * _spread(f4(448) / rr, n)
    if stochastic:
        # (values of the codes' subnormal range are held to 2^-30 before the bits are added)
        bits, near = ol.random16(seed, step, i, n) / 65536, np.where(y < 2.0 ** -6, 2.0 ** -30, 0)
        v = tuple(_rounded(np.maximum(y.astype(np.float64) + e, 0) + (e < 0) * (y > 0) * 2.0 ** -200, bits) for e in (-near, near))
    else:
        v = _nearest(np.where(r > 0, np.maximum(y, f4(2.0 ** -9)), y))
        v = (v, v)
    return _nearest(m * _spread(f4(448) / mm, n)), mm / f4(448), v, rr / f4(448)


def same(s, before, **kw):
    for i in range(len(s["params"])):
        m, m_scale, v, v_scale = expected(before, i, **kw)
        np.testing.assert_array_equal(_f32(s["m_scale"][i]), m_scale)
        np.testing.assert_array_equal(_f32(s["v_scale"][i]), v_scale)
        np.testing.assert_array_equal(_f32(s["m"][i]), m)
        got = _f32(s["v"][i])
        assert ((got >= v[0]) & (got <= v[1])).all()


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("ptype,off", [(BF, 0), (F32, 1)])
def test_clipped_steps(stochastic, ptype, off):
    """Norms and limits of every kind: the factor is that of fp64, rounded once."""
    rng = np.random.default_rng(5)
    s, moved = _state([1300, 129], True, ptype, seed=7, off=off), 0
    for step in range(1, 25):
        before = _copy(s)
        norm = float(np.exp(rng.uniform(-3, 3)))
        max_norm = norm * float(rng.uniform(0.3, 1.0))
        f = ol.clip_factor(norm * norm, max_norm)
        moved += f4(f) != f4(ol.clip_factor(norm * norm, float(f4(max_norm))))
        kw = dict(step=step, stochastic=stochastic, seed=11)
        mg.moe_adamw(**s, **HYPER, **kw, sumsq=torch.full((1,), norm * norm, dtype=torch.float64, device=DEV), max_norm=max_norm)
        same(s, before, f=f, **kw)
    assert moved > 0   # (some limits are not those of their fp32 values)


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("size", [1e-30, 1e-20, 1e-10, 1.0, 2e4, 4e4, 1e5, 1e9, 1e11, 1e12, 1e15, 1e18])
def test_roots_of_every_size(stochastic, size):
    """beta2 = 0: the root of v is the gradient's magnitude.  (That of the smallest
    is zero: its square leaves fp32.)"""
    n = 128 * 6 + 50
    s = _state([n, n], True, F32, seed=13, first=True)
    g = torch.Generator(DEV).manual_seed(3)
    for i, wide in enumerate((0.5, 3.0)):   # the second's codes reach the subnormal ones and the least one
        s["grads"][i].copy_(size * torch.exp(wide * torch.randn(n, generator=g, device=DEV)).clamp(max=10))
        s["grads"][i][::7] *= -1
        s["grads"][i][128:256:3] = 0
    before = _copy(s)
    kw = dict(step=3, stochastic=stochastic, seed=2, beta2=0.0)
    mg.moe_adamw(**s, **{**HYPER, **kw})
    same(s, before, **kw)
    root = _f32(s["v"][0]) * _spread(_f32(s["v_scale"][0]), n)
    want = np.abs(_f32(before["grads"][0])) if size > 1e-30 else np.zeros(n)
    ok = want > size * 0.05   # (whose codes are normal ones: within a step, an eighth)
    assert ok.sum() > n // 2 or size == 1e-30
    assert (np.abs(root - want)[ok] <= 0.126 * want[ok]).all()


@pytest.mark.parametrize("base,beta2", [(1.0, 0.5), (2.0, 0.25)])
def test_roots_of_every_significand(base, beta2):
    """One element of each block has a v in [1/2, 1) or [1, 2), so that the block's
    scale shows its root (a quotient of which is rounded once more)."""
    n, seen = 1 << 20, torch.zeros(1 << 23, dtype=torch.bool, device=DEV)
    first = torch.arange(n, device=DEV) * 128
    low = beta2 * base * base
    grads, codes, zeros = (torch.zeros(128 * n, dtype=t, device=DEV) for t in (F32, torch.uint8, torch.uint8))
    codes[first] = 0x38   # 1
    for part in range(8):
        k = torch.arange(part * n, (part + 1) * n, device=DEV, dtype=torch.float64)
        d = (k * 2.0 ** -23 * low / (1 - beta2)).sqrt().float()
        grads[first] = d
        m, v, ms, vs = zeros.clone(), codes.clone(), torch.ones(n, device=DEV), torch.full((n,), base, device=DEV)
        mg.moe_adamw(params=[torch.zeros(128 * n, dtype=BF, device=DEV)], grads=[grads], m=[m], v=[v], m_scale=[ms], v_scale=[vs], lr=0.0, beta1=0.0,
                     beta2=beta2)
        x = low + (1 - beta2) * d * d   # (fp32, each operation rounded)
        assert torch.equal(vs, (x.double().sqrt().float().double() / 448).float())
        seen[(x.view(torch.int32) & 0x7fffff).long()[x < 2 * low]] = True
    assert seen.float().mean() > 0.6


def test_root_of_the_significand_that_depends_on_the_hardware():
    """v = 0x406e9372 times 4^k (a half of a scale's square): the one root that an
    approximation within an ulp could spoil, by an ulp down.  The block's largest
    root makes it 11.5 before its code, a tie that goes to 12; an ulp less would
    go to 11."""
    k = torch.arange(-48, 58, device=DEV, dtype=torch.float64)
    n = len(k)
    scale, d = (torch.tensor(x, dtype=F32, device=DEV).double().mul(torch.exp2(k)).float() for x in (2.730476, 106.36985))
    grads, v = torch.zeros(128 * n, device=DEV), torch.zeros(128 * n, dtype=torch.uint8, device=DEV)
    v[::128] = 0x38   # 1
    grads[1::128] = d
    m, ms, vs = torch.zeros_like(v), torch.ones(n, device=DEV), scale.clone()
    mg.moe_adamw(params=[torch.zeros(128 * n, dtype=BF, device=DEV)], grads=[grads], m=[m], v=[v], m_scale=[ms], v_scale=[vs], lr=0.0, beta2=0.5)
    x = 0.5 * (scale * scale)
    assert ((x.view(torch.int32) & 0x7fffff) == 0x6e9372).all()
    largest = (0.5 * d * d).double().sqrt().float()
    r = x.double().sqrt().float()
    y = r * (448.0 / largest.double()).float()
    assert (y == 11.5).all() and (torch.nextafter(r, torch.zeros_like(r)) * (448.0 / largest.double()).float() < 11.5).all()
    assert torch.equal(vs, (largest.double() / 448).float())
    assert (v[::128].view(torch.float8_e4m3fn).float() == 12).all()
