"""The block-scaled FP8 layer (ExpertBlock, prec=PREC_FP8), its router's losses
and the clipping of its gradients, run together as a training step and as a
decoding step.

Every stage is held to the oracle on the operands the GPU itself stored:
codes bit-exact, products within the bound of their own sums (see
test_gpu_fp8), so that no stage hides behind another's rounding."""

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import moe as om
from oracle import numerics as nu
from oracle import step as st

from .gpu_util import dev_bf16

pytestmark = pytest.mark.gpu

DEV = "cuda"


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _host(t):
    return t.double().cpu().numpy()


def _inputs(E, H, N1, I, T, seed):
    rng = np.random.default_rng(seed)
    up = lambda v: dev_bf16(nu.f64_to_bf16_bits(nu.round_bf16(v)))
    w1, w2 = up(0.05 * rng.standard_normal((E, N1, H))), up(0.05 * rng.standard_normal((E, H, I)))
    logits = torch.from_numpy((rng.standard_normal((T, E)) + rng.standard_normal((1, E))).astype(np.float32)).to(DEV)
    return up(rng.standard_normal((T, H))), up(rng.standard_normal((T, H))), w1, w2, logits


def _product_check(blk, q, s, wq, ws, c, K, rows):
    sizes, starts = blk.split_sizes.tolist(), blk.padded_offsets.tolist()
    a = st.dequantize_rows(q.cpu().numpy()[:rows], s.cpu().numpy()[:, :rows])
    w = np.stack([st.dequantize_tiles(x, y) for x, y in zip(wq.cpu().numpy(), ws.cpu().numpy())])
    ref, mag = st.grouped_product(a, w, sizes, starts)
    got, ok = _host(c)[:rows], ~np.isnan(ref)
    tol = ((128 + -(-K // 128) + 4) * 2.0 ** -23 + 7 * 2.0 ** -13) * mag
    tol = tol + 2.0 ** -8 * (np.abs(np.nan_to_num(ref)) + tol)
    assert (np.abs(got - ref)[ok] <= tol[ok]).all()


def _rows_check(blk, name, x, rows, wgrad):
    """The stored copies are the encoding of the stored bf16 rows."""
    v = _host(x)[:rows]
    q, s = st.quantize_rows(v)
    np.testing.assert_array_equal(getattr(blk, name + "_q8").cpu().numpy()[:rows], q)
    np.testing.assert_array_equal(getattr(blk, name + "_s8").cpu().numpy()[:, :rows], s)
    if wgrad:
        q, s = st.quantize_rows(v.T.copy())
        np.testing.assert_array_equal(getattr(blk, name + "T_q8").cpu().numpy()[:, :rows], q)
        np.testing.assert_array_equal(getattr(blk, name + "T_s8").cpu().numpy()[:rows // 128], s)


CASES = [
    # E, k, T, H, I, act
    (4, 2, 256, 128, 256, mg.ACT_SWIGLU),
    (6, 3, 301, 192, 320, mg.ACT_GEGLU),
    (5, 2, 77, 320, 64, mg.ACT_SRELU),
    (8, 2, 8, 256, 192, mg.ACT_SWIGLU),      # decoding: at most 8 rows a group
    (8, 2, 1, 256, 192, mg.ACT_SWIGLU),
    (3, 1, 30, 128, 128, mg.ACT_SWIGLU),     # the second kernel for few rows
]


@pytest.mark.parametrize("wtype", [mg.TYPE_BF16, mg.TYPE_F32])
@pytest.mark.parametrize("E,k,T,H,I,act", CASES)
def test_step_stage_by_stage(E, k, T, H, I, act, wtype):
    blk = mg.ExpertBlock(E, H, I, T, k, act=mg.act_params(act), prec=mg.PREC_FP8, wgrad=True, wgrad_type=wtype)
    N1 = blk.N1
    x, dout, w1, w2, logits = _inputs(E, H, N1, I, T, E * T)
    blk.load_weights(w1, w2)
    blk.route_logits(logits)
    out = blk.forward(x, blk.expert_idx, blk.probs)
    losses = blk.router_loss(logits, balance_coef=0.1, z_coef=0.01).clone()
    dx, dprobs = blk.backward(dout)
    dlogits = blk.router_backward()
    dw1, dw2 = (g.clone() for g in blk.weight_grads())
    torch.cuda.synchronize()
    assert blk.err_flag.item() == 0
    rows = blk.padded_offsets[-1].item()
    sizes, starts = blk.split_sizes.tolist(), blk.padded_offsets.tolist()
    # weights
    for name, w in (("w1", blk.w1i), ("w2", blk.w2)):
        for e in range(E):
            q, s = st.quantize_tiles(_host(w[e]))
            for suffix, a, b in (("", q, s), ("t", q.T, s.T)):
                np.testing.assert_array_equal(getattr(blk, name + suffix + "_q8")[e].cpu().numpy(), a)
                np.testing.assert_array_equal(getattr(blk, name + suffix + "_s8")[e].cpu().numpy(), b)
    for name, t in (("xp", blk.xp), ("a", blk.a), ("dyp", blk.dyp), ("dz", blk.dz)):
        _rows_check(blk, name, t, rows, True)
    _product_check(blk, blk.xp_q8, blk.xp_s8, blk.w1_q8, blk.w1_s8, blk.z, H, rows)
    _product_check(blk, blk.a_q8, blk.a_s8, blk.w2_q8, blk.w2_s8, blk.yp, I, rows)
    _product_check(blk, blk.dyp_q8, blk.dyp_s8, blk.w2t_q8, blk.w2t_s8, blk.da, H, rows)
    _product_check(blk, blk.dz_q8, blk.dz_s8, blk.w1t_q8, blk.w1t_s8, blk.dxp, N1, rows)
    for left, right, dw in (("dz", "xp", dw1), ("dyp", "a", dw2)):
        ops = [st.dequantize_rows(getattr(blk, n + "T_q8").cpu().numpy()[:, :rows], getattr(blk, n + "T_s8").cpu().numpy()[:rows // 128])
               for n in (left, right)]
        ref, mag = st.grouped_weight_grad(*ops, sizes, starts)
        tol = 2 * (128 + rows // 128 + 4) * 2.0 ** -23 * mag
        if wtype == mg.TYPE_BF16:
            tol = tol + 7 * 2.0 ** -13 * mag
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert (np.abs(_host(dw) - ref) <= tol).all()
    if wtype == mg.TYPE_F32:   # a second micro-batch of the same step
        blk.weight_grads(accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(blk.dw1, dw1 + dw1) and torch.equal(blk.dw2, dw2 + dw2)
        blk.weight_grads()
    # the router's part
    counts, n, mean, loss = st.router_loss(logits.cpu().numpy(), blk.expert_idx.cpu().numpy(), None, 0.1, 0.01)
    np.testing.assert_array_equal(blk.router_counts.cpu().numpy(), counts)
    np.testing.assert_allclose(_host(losses), loss, rtol=800 * 2.0 ** -24)
    ref, scale = st.router_bwd(logits.cpu().numpy(), blk.expert_idx.cpu().numpy(), _host(dprobs), None, counts, n, None, 0.1, 0.01)
    assert (np.abs(_host(dlogits) - ref) <= 400 * 2.0 ** -24 * scale + 1e-37).all()
    # clipping, with the router's gradient among the others
    grads = [dw1.double(), dw2.double(), dlogits.double().clone()]
    norm = float(sum((g ** 2).sum() for g in grads)) ** 0.5
    got = blk.clip_grads(0.25 * norm, extra=[blk.dlogits])
    torch.cuda.synchronize()
    assert abs(got.item() - norm) <= 1e-6 * norm
    f = st.clip_factor(norm, 0.25 * norm)
    for g, o in zip(grads, (blk.dw1, blk.dw2, blk.dlogits)):
        # below the smallest normal number a rounding is off by an absolute half step
        tol = (g * f).abs() * ((2.0 ** -8 if o.dtype == torch.bfloat16 else 0) + 2.0 ** -21) + 2.0 ** -133
        assert int((~((o.double() - g * f).abs() <= tol)).sum()) == 0


def test_empty_experts_and_live_only_weights():
    """All tokens to two of six experts: the others' gradients are zero and,
    with live_only, their weight copies stay as they were."""
    E, k, T, H, I = 6, 2, 50, 128, 192
    blk = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8, wgrad=True)
    x, dout, w1, w2, _ = _inputs(E, H, 2 * I, I, T, 3)
    blk.load_weights(w1, w2)
    idx = torch.tensor([[1, 4]] * T, dtype=torch.int32, device=DEV)
    probs = torch.full((T, k), 0.5, device=DEV)
    blk.w1_q8.fill_(0x11)
    blk.route(idx, probs, x)
    blk.quantize_weights(live_only=True)
    blk.experts_forward_fp8()
    blk.combine(blk.yp, blk.out)
    blk.backward(dout)
    blk.weight_grads()
    torch.cuda.synchronize()
    for e in range(E):
        live = e in (1, 4)
        assert bool(blk.dw1[e].any()) == live and bool(blk.dw2[e].any()) == live
        assert bool((blk.w1_q8[e] != 0x11).any()) == live
    assert torch.isfinite(blk.out.float()).all()


def test_share_of_the_experts():
    """Two blocks with half of the experts each: their outputs add up to the
    whole layer's (one bf16 rounding each), dprobs are the whole's exactly."""
    E, k, T, H, I = 8, 2, 120, 128, 128
    x, dout, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 4)
    whole = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8)
    whole.load_weights(w1, w2)
    whole.route_logits(logits)
    out = whole.forward(x, whole.expert_idx, whole.probs).float()
    dprobs = whole.backward(dout)[1]
    parts = []
    for first in (0, 4):
        b = mg.ExpertBlock(4, H, I, T, k, first_expert=first, prec=mg.PREC_FP8)
        b.load_weights(w1[first:first + 4].contiguous(), w2[first:first + 4].contiguous())
        parts.append((b.forward(x, whole.expert_idx, whole.probs).float(), b.backward(dout)[1].clone(), b.yp.float().abs().max()))
    torch.cuda.synchronize()
    both = parts[0][0] + parts[1][0]
    # three bf16 roundings (two parts, the whole) of numbers up to k yp's
    assert ((both - out).abs() <= 3 * 2.0 ** -8 * k * max(parts[0][2], parts[1][2])).all()
    assert torch.equal(parts[0][1] + parts[1][1], dprobs)


def test_refusals():
    for kw in (dict(recompute=True), dict(unfused=True)):
        with pytest.raises(ValueError):
            mg.ExpertBlock(4, 128, 128, 16, 2, prec=mg.PREC_FP8, **kw)
    with pytest.raises(ValueError):
        mg.ExpertBlock(4, 128, 128, 16, 2, wgrad=True, wgrad_type=mg.TYPE_F32)
    blk = mg.ExpertBlock(4, 128, 128, 16, 2, prec=mg.PREC_FP8)
    x, dout, w1, w2, logits = _inputs(4, 128, 256, 128, 16, 5)
    with pytest.raises(RuntimeError):
        blk.router_backward()
    with pytest.raises(ValueError):   # picks of other tokens than the logits'
        blk.router_loss(logits, expert_idx=torch.zeros(15, 2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        blk.router_loss(logits, expert_idx=torch.zeros(16, 4, dtype=torch.int32, device=DEV))
    blk.router_loss(logits, expert_idx=torch.zeros(16, 2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        blk.router_backward(dprobs=torch.zeros(16, 4, device=DEV))
    # logits of another batch: outputs of that size
    blk.router_loss(logits[:5].clone(), expert_idx=torch.zeros(5, 2, dtype=torch.int32, device=DEV))
    assert blk.router_backward(dprobs=torch.zeros(5, 2, device=DEV)).shape == (5, 4)
    for f in (blk.weight_grads, lambda: blk.clip_grads(1.0)):
        with pytest.raises(RuntimeError):
            f()
    blk.load_weights(w1, w2, bias1=torch.zeros(4, 256, device=DEV))
    blk.route_logits(logits)
    with pytest.raises(RuntimeError):
        blk.forward(x, blk.expert_idx, blk.probs)
    blk = mg.ExpertBlock(4, 128, 128, 16, 2, prec=mg.PREC_FP8, wgrad=True)
    with pytest.raises(RuntimeError):
        blk.weight_grads(accumulate=True)


def test_whole_step_in_a_graph():
    E, k, T, H, I = 8, 2, 200, 256, 320
    blk = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8, wgrad=True)
    x, dout, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 6)
    blk.load_weights(w1, w2)
    names = ("out", "dx", "dprobs", "dw1", "dw2", "dlogits", "router_losses", "router_counts", "grad_norm")

    def step():
        blk.route_logits(logits, x)
        blk.quantize_weights(live_only=True)
        blk.experts_forward_fp8()
        blk.combine(blk.yp, blk.out)
        blk.router_loss(logits, balance_coef=0.1, z_coef=0.01)
        blk.backward(dout)
        blk.router_backward()
        blk.weight_grads()
        blk.clip_grads(1.0, extra=[blk.dlogits])

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in range(3):
        nx, nd, _, _, nl = _inputs(E, H, 2 * I, I, T, 10 + seed)
        x.copy_(nx); dout.copy_(nd); logits.copy_(nl)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [getattr(blk, n).clone() for n in names]
        step()
        torch.cuda.synchronize()
        for n, g in zip(names, got):
            assert torch.equal(g, getattr(blk, n)), n


def test_buffers_of_a_captured_graph_survive_other_shapes():
    """A graph captured with one shape of logits and list of gradients writes
    the same buffers after eager calls with others."""
    E, k, T, H, I = 8, 2, 96, 128, 128
    blk = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8, wgrad=True)
    x, dout, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 7)
    blk.load_weights(w1, w2)
    blk.route_logits(logits)
    blk.forward(x, blk.expert_idx, blk.probs)
    blk.backward(dout)
    blk.weight_grads()

    def tail():
        blk.router_loss(logits, balance_coef=0.1, z_coef=0.01)
        blk.router_backward()
        blk.clip_grads(1e9, extra=[blk.dlogits])

    tail()
    mine = [blk.dlogits, blk.router_losses, blk.grad_norm]
    want = [t.clone() for t in mine]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tail()
    few = torch.randn(33, E, device=DEV)
    many = [torch.ones(1000 + i, device=DEV) for i in range(200)]
    blk.router_loss(few, expert_idx=torch.zeros(33, k, dtype=torch.int32, device=DEV))
    blk.clip_grads(1e9, extra=many)
    other = [torch.full((n,), 7.0, device=DEV) for n in (T * E, T * E, 2, 2, 64, 1024, 4096)]   # what a freed buffer would become
    for t in mine:
        t.fill_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(mine, want):
        assert torch.equal(a, b)
    assert all(bool((o == 7.0).all()) for o in other)
    blk.router_loss(logits)
    assert blk.dlogits is mine[0]
