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
