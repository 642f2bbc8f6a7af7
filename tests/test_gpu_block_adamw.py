"""ExpertBlock's AdamW steps between loads, graphs and checkpoints."""

import gc

import pytest
import torch

import moe_grouped_mlp_amd as mg

from .test_gpu_fp8_block import _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
E, H, I, T, K = 4, 128, 128, 32, 2


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """Tests after these measure what torch's allocator holds."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _block(seed):
    _, _, w1, w2, _ = _inputs(E, H, 2 * I, I, T, seed)
    blk = mg.ExpertBlock(E, H, I, T, K, wgrad=True)
    blk.load_weights(w1, w2)
    return blk, w1, w2


def _grads(blk, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    for dw in (blk.dw1, blk.dw2):
        dw.copy_(torch.randn(dw.shape, generator=g, device=DEV))


def _states(blk):
    st = blk._adamw
    return [blk.w1i, blk.w2, *st["m"], *st["v"], *(st["m_scale"] or ()), *(st["v_scale"] or ()), *(st["master"] or ())]


def _equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(_states(a), _states(b)))


@pytest.mark.parametrize("state,master", [(mg.STATE_F32, True), (mg.STATE_FP8, False)])
def test_a_captured_step_goes_on_after_load_weights(state, master):
    """Replays after other weights were loaded are the first steps from those, as
    an eager block makes them."""
    kw = dict(weight_decay=0.1, max_norm=3.0, state=state, master=master, stochastic=state == mg.STATE_FP8, seed=1, capturable=True)
    blk, *_ = _block(1)
    _grads(blk, 0)
    blk.adamw_step(1e-2, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.adamw_step(1e-2, **kw)
    graph.replay()
    other, w1, w2 = _block(2)
    blk.load_weights(w1, w2)
    spare = [torch.full_like(t, 3) for t in _states(blk)]   # (memory given back would be these now)
    for step in range(3):
        _grads(blk, step)
        _grads(other, step)
        graph.replay()
        other.adamw_step(1e-2, **kw)
        torch.cuda.synchronize()
        assert _equal(blk, other) and blk._adamw["step"].item() == step + 1
    assert all((t == 3).all() for t in spare)
    blk.adamw_step(1e-2, **kw)   # and an eager one after them
    other.adamw_step(1e-2, **kw)
    assert _equal(blk, other)


def test_norm_over_other_gradients():
    """A step with the router's gradient in the norm is the step of gradients that
    clip_grads() scaled with it.  (It rounds them to bf16, 2^-8; the update of a first step
    hardly depends on their size: its error is that of eps beside their root.)"""
    blk, *_ = _block(3)
    two, *_ = _block(3)
    extra = torch.randn(300, device=DEV)
    for b in (blk, two):
        _grads(b, 4)
    kept = extra.clone()
    blk.adamw_step(1e-2, max_norm=1.0, extra=[extra], beta1=0.0, beta2=0.0, eps=1.0)
    norm = two.clip_grads(1.0, extra=[extra])
    assert torch.equal(blk.grad_sumsq, two.grad_sumsq) and abs(blk.grad_sumsq.sqrt().item() - norm.item()) <= 2.0 ** -23 * norm.item()
    assert blk.grad_sumsq.item() > (blk.dw1.double().square().sum() + blk.dw2.double().square().sum() + kept.double().square().sum()).item() * (1 - 1e-12)
    two.adamw_step(1e-2, beta1=0.0, beta2=0.0, eps=1.0)
    for a, b, w, g in zip(blk._adamw["master"], two._adamw["master"], (blk.w1i, blk.w2), (two.dw1, two.dw2)):
        assert ((a - b).abs() <= 1e-2 * 2.0 ** -8 * 1.01 * g.float().abs().view(-1) + 2.0 ** -22 * a.abs()).all()
    given, *_ = _block(3)
    _grads(given, 4)
    given.adamw_step(1e-2, max_norm=1.0, sumsq=blk.grad_sumsq, beta1=0.0, beta2=0.0, eps=1.0)
    assert _equal(blk, given)


@pytest.mark.parametrize("kw", [dict(), dict(state=mg.STATE_FP8, master=False, stochastic=True, seed=2), dict(capturable=True)])
def test_resumed_steps(kw, tmp_path):
    """A block that goes on from a file is the block that wrote it, bit for bit."""
    blk, *_ = _block(5)
    for step in range(2):
        _grads(blk, step)
        blk.adamw_step(1e-2, **kw)
    w1, w2 = torch.empty_like(blk.w1i), blk.w2.clone()
    mg.moe_weight_repack_interleave(blk.w1i, w1, E, I, H, inverse=True)
    torch.save(dict(w1=w1, w2=w2, adamw=blk.adamw_state()), tmp_path / "state.pt")
    for step in (2, 3):
        _grads(blk, step)
        blk.adamw_step(1e-2, **kw)
    saved = torch.load(tmp_path / "state.pt", weights_only=True)
    other, *_ = _block(6)
    other.load_weights(saved["w1"], saved["w2"])
    other.load_adamw_state(saved["adamw"])
    for step in (2, 3):
        _grads(other, step)
        other.adamw_step(1e-2, **kw)
    assert _equal(blk, other)
