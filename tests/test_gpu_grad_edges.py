"""Gradient clipping at its edges."""

import pytest
import torch

import moe_grouped_mlp_amd as mg

from .test_gpu_grad import _make, _sumsq

pytestmark = pytest.mark.gpu


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


@pytest.mark.parametrize("at", [0, 17, 2999])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_copies_of_gradients_whose_norm_is_not_finite(bad, at):
    """Out of place, every number is copied with its bits and a NaN stays one."""
    grads = _make([100, 3000, 1001])
    grads[1][at] = bad
    s = _sumsq(grads)
    out = [torch.full_like(g, 5.0) for g in grads]
    mg.moe_grad_clip(tensors=grads, out=out, sumsq=s, max_norm=1e-3)
    torch.cuda.synchronize()
    for g, o in zip(grads, out):
        bits = torch.int16 if g.dtype == torch.bfloat16 else torch.int32
        number = ~torch.isnan(g)
        assert torch.equal(g.view(bits)[number], o.view(bits)[number])
        assert torch.equal(torch.isnan(o), ~number)
