"""What ExpertBlock keeps of the router by scores between calls (no GPU needed: the
library's calls are replaced by ones that do nothing, the buffers are host tensors)."""

import unittest.mock as mock

import pytest
import torch

import moe_grouped_mlp_amd as mg
from moe_grouped_mlp_amd import binding as B
from moe_grouped_mlp_amd import block as blk_mod

E, H, I, T, K = 4, 128, 128, 16, 2
CALLS = ("moe_permute", "moe_unpermute", "moe_quantize_fp8", "moe_grouped_gemm_fp8", "moe_glu_unfused", "moe_router_route",
         "moe_router_topk", "moe_router_gate", "moe_router_gate_bwd", "moe_router_bias_update")


@pytest.fixture
def block():
    with mock.patch.multiple(B, **{n: lambda **kw: None for n in CALLS}):
        yield mg.ExpertBlock(E, H, I, T, K, prec=mg.PREC_FP8, device="cpu")


def _x():
    return torch.zeros(T, H, dtype=torch.bfloat16)


def test_gate_backward_takes_its_own_picks_gradients_only(block):
    logits, x, dprobs = torch.zeros(T, E), _x(), torch.zeros(T, K)
    with pytest.raises(RuntimeError, match="gate"):
        block.gate_backward(dprobs)
    block.gate(logits)
    with pytest.raises(RuntimeError, match="backward"):
        block.gate_backward()   # none yet
    block.forward(x, block.expert_idx, block.probs)
    block.backward(x)
    with mock.patch.object(B, "moe_router_gate_bwd") as bwd:
        block.gate_backward()
        assert bwd.call_args.kwargs["dprobs"] is block.dprobs and bwd.call_args.kwargs["logits"] is logits
    # rows routed by other picks: their gradients are not those of gate()'s
    block.forward(x, torch.zeros(T, K, dtype=torch.int32), block.probs)
    block.backward(x)
    with pytest.raises(RuntimeError, match="picks"):
        block.gate_backward()
    block.gate_backward(dprobs)   # given ones are taken
    block.forward(x, block.expert_idx, block.probs)
    block.backward(x)
    block.gate_backward()


@pytest.mark.parametrize("fused", [False, True])
def test_gate_backward_after_another_router(block, fused):
    """route_logits() writes its picks over gate()'s."""
    block.gate(torch.zeros(T, E))
    block.route_logits(torch.zeros(T, E), fused=fused)
    block.forward(_x(), block.expert_idx, block.probs)
    block.backward(_x())
    for given in (None, torch.zeros(T, K)):
        with pytest.raises(RuntimeError, match="route_logits"):
            block.gate_backward(given)
    block.update_bias(torch.zeros(E), 0.1)   # its counts are still there


def test_a_capture_makes_no_counters(block):
    """Their clearing would be part of every replay."""
    with mock.patch.object(blk_mod, "_capturing", lambda t: True):
        with pytest.raises(RuntimeError, match="captured"):
            block.gate(torch.zeros(T, E), count=True)
    block.gate(torch.zeros(T, E), count=True)
    counts = block.gate_counts
    block.gate(torch.zeros(T, 2 * E), count=True)
    with mock.patch.object(blk_mod, "_capturing", lambda t: True):
        block.gate(torch.zeros(T, E), count=True)
    assert block.gate_counts is counts
