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
    with mock.patch.multiple(B, **{n: lambda **kw: None for n in CALLS}):   # (a Mock would hold what it is given)
        yield mg.ExpertBlock(E, H, I, T, K, prec=mg.PREC_FP8, device="cpu")


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
    with mock.patch.object(B, "moe_router_bwd") as bwd:
        block.router_backward()
        assert bwd.call_args.kwargs["dprobs"] is block.dprobs
    block.router_backward()     # again, say for a graph's warm-up
    block.forward(x, _idx(), probs)
    refused()
    block.backward(x)
    for fused in (False, True):
        block.route_logits(logits, fused=fused)
        refused()
        block.backward(x)
        block.router_backward()


def _sizes_alive(refs):
    gc.collect()
    return sum(r() is not None for r in refs)


def _loss(block, n, hold=None):
    block.router_loss(torch.zeros(n, E), expert_idx=_idx(n))
    for name in ("dlogits", "router_losses", "ws_loss"):
        if hold is not None:
            hold.append(weakref.ref(getattr(block, name)))


def test_router_buffers_do_not_pile_up(block):
    """A token count that differs from step to step keeps one shape's buffers."""
    refs = []
    for n in range(1, 200):
        _loss(block, n, refs)
    assert _sizes_alive(refs) == 3
    assert block.dlogits.shape == (199, E)


def test_router_buffers_of_captured_graphs_stay(block):
    """Shapes that a capture used are kept, whether their buffers were made in
    it or before, and are found again; the others are not."""
    warm, captured = [], []
    _loss(block, 7, warm)
    before = block.dlogits
    with mock.patch.object(blk_mod, "_capturing", lambda t: True):
        _loss(block, 7)
        assert block.dlogits is before
        _loss(block, 9, captured)
    for n in range(20, 60):
        _loss(block, n)
    assert _sizes_alive(warm) == 3 and _sizes_alive(captured) == 3
    _loss(block, 7)
    assert block.dlogits is before
    _loss(block, 9)
    assert captured[0]() is block.dlogits


def test_results_held_by_the_caller_stay(block):
    """A returned tensor is the caller's as long as it holds it."""
    losses = block.router_loss(torch.zeros(5, E), expert_idx=_idx(5))
    losses.fill_(3.0)
    block.router_loss(torch.zeros(6, E), expert_idx=_idx(6)).fill_(4.0)
    assert losses.tolist() == [3.0, 3.0]


def test_other_streams_than_the_buffers_own_are_recorded(block):
    """Memory that a call on another stream than the buffers' own uses is not
    given back under that stream."""
    seen = []
    stream = mock.Mock(side_effect=lambda: 1)
    with mock.patch.object(blk_mod, "_stream_of", lambda t: stream()), \
            mock.patch.object(blk_mod, "_record", lambda t: seen.append(t)):
        _loss(block, 5)
        _loss(block, 5)
        assert not seen
        stream.side_effect = lambda: 2
        _loss(block, 5)
        names = ("router_counts", "router_tokens", "router_prob_mean", "router_losses", "dlogits", "ws_loss")
        assert {id(t) for t in seen} == {id(getattr(block, n)) for n in names}
        seen.clear()
        block.router_backward(dprobs=torch.zeros(5, K))
        assert not seen     # once is enough for a stream
        stream.side_effect = lambda: 3
        block.router_backward(dprobs=torch.zeros(5, K))
        assert id(block.dlogits) in {id(t) for t in seen}
