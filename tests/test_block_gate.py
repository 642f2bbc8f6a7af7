"""What ExpertBlock keeps of the router by scores when calls are refused, and with
routers of several sizes (no GPU needed: the library's calls are replaced by ones that
do nothing, the buffers are host tensors)."""

import unittest.mock as mock

import pytest
import torch

import moe_grouped_mlp_amd as mg
from moe_grouped_mlp_amd import binding as B

from .test_block_layer_steps import CALLS, E, H, I, K, T, _x


@pytest.fixture
def block():
    with mock.patch.multiple(B, **{n: lambda **kw: None for n in CALLS}):
        yield mg.ExpertBlock(E, H, I, T, K, prec=mg.PREC_FP8, device="cpu")


def _refuse(**kw):
    raise mg.MoeError("moe_router_gate", 1, "no")


def test_a_refused_gate_changes_nothing(block):
    """The picks that are there are those of the call before, and so are the logits
    and the kind of scores that gate_backward() takes for them."""
    logits = torch.zeros(T, E)
    block.gate(logits, renorm=True, count=True)
    counts = block.gate_counts
    block.forward(_x(), block.expert_idx, block.probs)
    block.backward(_x())
    with mock.patch.object(B, "moe_router_gate", _refuse), pytest.raises(mg.MoeError):
        block.gate(torch.ones(T, 2 * E), score=mg.SCORE_SIGMOID, scale=float("nan"), count=True)
    assert block.gate_counts is counts
    with mock.patch.object(B, "moe_router_gate_bwd") as bwd:
        block.gate_backward()
    kw = bwd.call_args.kwargs
    assert kw["logits"] is logits and kw["E"] == E and kw["renorm"] is True and kw["score"] == mg.SCORE_SOFTMAX and kw["scale"] == 1.0


def test_a_refused_first_gate_leaves_nothing(block):
    with mock.patch.object(B, "moe_router_gate", _refuse), pytest.raises(mg.MoeError):
        block.gate(torch.zeros(T, E), count=True)
    with pytest.raises(RuntimeError, match="gate"):
        block.gate_backward(torch.zeros(T, K))
    with pytest.raises(RuntimeError, match="gate"):
        block.update_bias(torch.zeros(E), 0.1)


def test_bias_updates_of_two_routers(block):
    """Each bias goes by the counts of its own number of experts, in any order."""
    block.gate(torch.zeros(T, E), count=True)
    few = block.gate_counts
    block.gate(torch.zeros(T, 2 * E), count=True)
    many = block.gate_counts
    for size, counts in ((E, few), (2 * E, many)):
        block.gate(torch.zeros(T, 3 * E - size))   # (the other one was the last)
        with mock.patch.object(B, "moe_router_bias_update") as update:
            block.update_bias(torch.zeros(size), 0.1)
        assert update.call_args.kwargs["counts"] is counts and update.call_args.kwargs["E"] == size
