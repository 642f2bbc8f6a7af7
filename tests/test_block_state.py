"""What ExpertBlock keeps between calls (no GPU needed: the library's calls are
replaced by ones that do nothing, the block's buffers are host tensors)."""

import gc
import unittest.mock as mock
import weakref

import pytest
import torch

import moe_grouped_mlp_amd as mg
from moe_grouped_mlp_amd import binding as B
from moe_grouped_mlp_amd import block as blk_mod

E, H, I, T, K = 4, 128, 128, 16, 2
CALLS = ("moe_permute", "moe_unpermute", "moe_quantize_fp8", "moe_grouped_gemm_fp8", "moe_glu_unfused", "moe_router_route",
         "moe_router_topk", "moe_router_loss", "moe_router_bwd")


@pytest.fixture
def block():
    with mock.patch.multiple(B, **{n: mock.DEFAULT for n in CALLS}) as calls:
        b = mg.ExpertBlock(E, H, I, T, K, prec=mg.PREC_FP8, device="cpu")
        b.calls = calls
        yield b


def _idx(n=T):
    return torch.zeros(n, K, dtype=torch.int32)


def test_router_backward_refuses_dprobs_of_an_earlier_step(block):
    """Without dprobs given they are those of a backward() since the last
    route(): none before the first one, none of the step before."""
    logits, x, probs = torch.zeros(T, E), torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, K)

    def refused():
        block.router_loss(logits, expert_idx=_idx())
        with pytest.raises(RuntimeError, match="backward"):
            block.router_backward()
        block.router_backward(dprobs=torch.zeros(T, K))   # given ones are taken

    refused()
    block.forward(x, _idx(), probs)
    refused()
    block.backward(x)
    block.router_loss(logits, expert_idx=_idx())
    block.router_backward()
    assert block.calls["moe_router_bwd"].call_args.kwargs["dprobs"] is block.dprobs
    block.router_backward()     # again, say for a graph's warm-up
    block.forward(x, _idx(), probs)
    refused()
    block.backward(x)
    for fused in (False, True):
        block.route_logits(logits, fused=fused)
        refused()
        block.backward(x)
        block.router_backward()
