"""The router losses' sums over tokens are made in fp64: the mean of equal
numbers is that number.  What stands in tokens that the mask leaves out reaches
nothing."""

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg

from .test_gpu_router_loss import _bwd, _loss

pytestmark = pytest.mark.gpu


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


@pytest.mark.parametrize("T,E,k", [(77, 3, 1), (1000, 8, 2), (4099, 60, 4), (3001, 256, 8), (30011, 8, 2), (7001, 1000, 8)])
def test_equal_tokens_have_their_own_mean(T, E, k):
    """T tokens of the same logits: n v / n in fp64 is v to 2^-52, so the mean
    probabilities and the z loss round to those of one token."""
    x = np.random.default_rng(E).standard_normal((1, E)).astype(np.float32)
    idx = np.argsort(-x, axis=1)[:, :k].astype(np.int32)
    one = _loss(x, idx, None, 0.0, 1.0)[1]
    all_ = _loss(np.repeat(x, T, 0), np.repeat(idx, T, 0), None, 0.0, 1.0)[1]
    assert torch.equal(all_["prob_mean"], one["prob_mean"])
    assert torch.equal(all_["loss"], one["loss"])


@pytest.mark.parametrize("E", [3, 30, 250])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_tokens_without_gradients_get_zeros(bad, E):
    """Padding may hold anything: a token that the mask leaves out, with no
    gradient of its own, gets zeros; with one the formula holds."""
    T, k = 50, 2
    rng = np.random.default_rng(3)
    x = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-x, axis=1)[:, :k].astype(np.int32)
    mask = np.ones(T, np.uint8)
    mask[40:] = 0
    x[40:, 1] = bad
    x[45:] = bad
    lg, out = _loss(x, idx, mask, 0.3, 0.2)
    assert out["n_tokens"].item() == 40 and torch.isfinite(out["loss"]).all()
    d = _bwd(lg, idx, mask, 0.3, 0.2, out)
    assert np.isfinite(d).all() and d[:40].any() and not d[40:].any()
    dprobs = rng.standard_normal((T, k)).astype(np.float32)
    dprobs[40:] = 0.0
    d = _bwd(lg, idx, mask, 0.3, 0.2, out, dprobs)
    assert np.isfinite(d).all() and not d[40:].any()
    bad_idx = idx.copy()
    bad_idx[42] = E + 1     # dropped picks: their gradients go nowhere
    other = dprobs.copy()
    other[42] = 1.0
    d = _bwd(lg, bad_idx, mask, 0.3, 0.2, out, other)
    assert np.isfinite(d).all() and not d[40:].any()
    dprobs[41, 0] = 1.0
    d = _bwd(lg, idx, mask, 0.3, 0.2, out, dprobs)
    assert np.isnan(d[41]).any() and np.isfinite(np.delete(d, 41, 0)).all()
