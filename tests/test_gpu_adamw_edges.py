"""AdamW (moe_adamw) at the ends of fp32's range, against the float64 oracle."""

import gc

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg

from .test_gpu_adamw import BF, DEV, F32, _np, _state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """Tests after these measure what torch's allocator holds."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("ptype", [BF, F32])
@pytest.mark.parametrize("size", [1e-16, 1e-18, 1e-19, 1e-20])
def test_no_eps_and_tiny_gradients(off, ptype, size):
    """The first step's update is lr times the gradient's sign, also where v is below fp32's
    normal numbers.  v = a d^2 is off by half of 2^-149, so its root by 2^-150 / v of itself,
    and the other steps are off by less than 2^-19."""
    n = 1000
    s = _state([n], False, ptype, F32, first=True, off=off)
    sign = torch.where(torch.arange(n, device=DEV) % 3 == 0, -1.0, 1.0)
    s["grads"][0].copy_(size * sign * torch.linspace(1, 2, n, device=DEV))
    s["params"][0].zero_()
    mg.moe_adamw(**s, lr=1.0, beta1=0.9, beta2=0.95, eps=0.0, step=1)
    d = _np(s["grads"][0])
    tol = 2.0 ** -150 / (0.05 * d * d) + 2.0 ** -19 + (2.0 ** -8 if ptype == BF else 0)
    assert (np.abs(_np(s["params"][0]) + np.sign(d)) <= 1.01 * tol).all()
