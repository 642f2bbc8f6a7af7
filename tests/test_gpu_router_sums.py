"""The router losses' sums over tokens are made in fp64: the mean of equal
numbers is that number."""

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg

from .test_gpu_router_loss import _loss

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
