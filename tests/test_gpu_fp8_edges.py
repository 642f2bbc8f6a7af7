"""Calls of the block-scaled FP8 layer at their edges."""

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import numerics as nu
from oracle import step as st

from .test_gpu_fp8 import (DEV, _check, _margin, _operands, _product, _reference, _starts, _wgrad, _wgrad_operands,
                           _wgrad_ref)
from .test_gpu_fp8_block import _inputs

pytestmark = pytest.mark.gpu


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def test_accumulation_leaves_empty_experts_as_they_are():
    """An expert with no rows adds nothing: not even the sign of a zero or a
    NaN's bits change."""
    sizes, P, Q = [0, 130, 0, 1, 0], 272, 144
    starts = _starts(sizes)
    ops = _wgrad_operands(np.random.default_rng(1), sizes, starts, starts[-1] + 128, P, Q, exact=True)
    ref, _ = _wgrad_ref(*ops, sizes, starts)
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (5, P, Q), dtype=torch.int32, device=DEV,
                         generator=torch.Generator(DEV).manual_seed(1))
    bits[0] = -2 ** 31      # -0
    bits[2, 0] = 0x7F800001  # a signalling NaN
    c = bits.view(torch.float32).clone()
    c[[1, 3]] = 3.0
    _wgrad(*ops, sizes, starts, c=c, accumulate=True)
    for e in (0, 2, 4):
        assert torch.equal(c[e].view(torch.int32), bits[e]), e
    np.testing.assert_array_equal(c[[1, 3]].double().cpu().numpy(), ref[[1, 3]] + 3.0)


@pytest.mark.parametrize("hint", [1, 16, 20, 32])
def test_few_rows_leave_the_margin_free(hint):
    """With a cu_margin products of few rows run on one workgroup a CU, as all
    others do: the tiled kernel, whose sums over K are in its own order."""
    sizes, N, K = [3, 0, 16, 1, 20], 272, 1168
    starts = _starts(sizes)
    ops = _operands(np.random.default_rng(2), sizes, starts, starts[-1], N, K)
    tiled = _product(*ops, sizes, starts, cu_margin=_margin(40))
    assert torch.equal(_product(*ops, sizes, starts, max_rows=hint, cu_margin=_margin(40)), tiled)
    few = _product(*ops, sizes, starts, max_rows=hint)
    assert not torch.equal(few, tiled)   # the other kernel, or this test shows nothing


@pytest.mark.parametrize("mode", [mg.QUANT_ROW, mg.QUANT_COL, mg.QUANT_BOTH, mg.QUANT_TILE])
def test_quantize_of_empty_tensors(mode):
    u8 = dict(dtype=torch.uint8, device=DEV)
    x = torch.empty(0, 48, dtype=torch.bfloat16, device=DEV)
    s = torch.empty(1, 0, device=DEV)
    mg.moe_quantize_fp8(mode=mode, batch=1, rows=0, cols=48, x=x, q=torch.empty(0, 48, **u8), s=s,
                        qT=torch.empty(48, 0, **u8), sT=torch.empty(0, 48, device=DEV))
    torch.cuda.synchronize()


def test_router_gradient_of_two_shares():
    """Two shares of a layer, the losses' gradient taken in one of them: their
    dlogits add up to the whole layer's, each off by its roundings."""
    E, k, T, H, I = 8, 2, 120, 128, 128
    x, dout, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 4)
    whole = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8)
    whole.load_weights(w1, w2)
    whole.route_logits(logits)
    idx, probs = whole.expert_idx, whole.probs

    def step(b, dloss=None):
        b.forward(x, idx, probs)
        b.backward(dout)
        b.router_loss(logits, expert_idx=idx, balance_coef=0.5, z_coef=0.1)
        return b.router_backward(dloss).double().cpu().numpy()

    want = step(whole)
    parts = []
    for first, dloss in ((0, None), (4, torch.zeros(2, device=DEV))):
        b = mg.ExpertBlock(4, H, I, T, k, first_expert=first, prec=mg.PREC_FP8)
        b.load_weights(w1[first:first + 4].contiguous(), w2[first:first + 4].contiguous())
        parts.append(step(b, dloss))
    _, scale = st.router_bwd(logits.cpu().numpy(), idx.cpu().numpy(), whole.dprobs.double().cpu().numpy(), None,
                             whole.router_counts.cpu().numpy(), T, None, 0.5, 0.1)
    # 400 half steps of the terms' magnitudes for each of the three
    assert (np.abs(parts[0] + parts[1] - want) <= 3 * 400 * 2.0 ** -24 * scale).all()


def test_router_losses_of_many_shapes_and_streams():
    """Steps of other token counts, now and then on another stream, around a
    graph captured with one: all give the results of a block of their own, and
    the memory of earlier shapes is given back."""
    E, k, T, H, I = 64, 2, 16, 128, 128
    blk = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8)
    logits = torch.randn(4096, E, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    idx = logits.topk(k, dim=1).indices.to(torch.int32)
    zeros = torch.zeros(4096, k, device=DEV)

    def step(b, n):
        losses = b.router_loss(logits[:n], expert_idx=idx[:n], balance_coef=0.5, z_coef=0.1)
        return losses, b.router_backward(dprobs=zeros[:n])

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step(blk, 1000)
    base = torch.cuda.memory_allocated()
    for i in range(60):
        n = 4096 - 50 * i
        with torch.cuda.stream(side if i % 3 == 1 else torch.cuda.current_stream()):
            got = [t.clone() for t in step(blk, n)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for m, have in ((n, got), (1000, held)):
            want = step(mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8), m)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(have, want)), (i, m)
        del got, have, want
        # one shape's gradient (1 MB at most) and workspace (at most 256 of 12 (E + 1) bytes)
        assert torch.cuda.memory_allocated() - base < 4 * 4096 * E + 256 * 12 * (E + 1) + (1 << 16), i


# ----------------------------------------- K cut with tiles of every width ---
@pytest.mark.parametrize("leave", [48, 80])
@pytest.mark.parametrize("c_type,fast", [(mg.TYPE_F32, False), (mg.TYPE_BF16, False), (mg.TYPE_BF16, True)])
@pytest.mark.parametrize("sizes", [[40, 0, 1], [100, 256, 65], [170, 0, 300], [250, 129, 0]])
def test_product_cut_along_k_every_tile_width(sizes, c_type, fast, leave):
    """A row buffer far larger than the routed rows and few CUs: the tiles are
    wide (two groups of 64 tokens, with fp8_sums and 48 CUs four), few, and K is
    cut; a group's last tile holds one to four groups.  Exact on integers; on
    random data the order of the parts shows."""
    N, K, M_cap = 272, 4112, 4096
    rng = np.random.default_rng(leave + len(sizes))
    starts = _starts(sizes)
    kw = dict(cu_margin=_margin(leave), fp8_sums=fast)
    assert mg.moe_grouped_gemm_fp8_workspace_size(len(sizes), N, K, M_cap, 0) > 0

    def padded(ops):
        a_q, a_s = np.full((M_cap, K), 0x7F, np.uint8), np.full((ops[1].shape[0], M_cap), np.nan, np.float32)
        a_q[:starts[-1]], a_s[:, :starts[-1]] = ops[0], ops[1]
        return a_q, a_s, *ops[2:]

    ops = _operands(rng, sizes, starts, starts[-1], N, K, exact=True)
    # one scale for all, and so few bits that every sum is exact
    ops = (nu.e4m3_encode(np.clip(np.nan_to_num(nu.e4m3_decode(ops[0])), -3, 3)), np.ones_like(ops[1]),
           nu.e4m3_encode(np.clip(nu.e4m3_decode(ops[2]), -3, 3)), np.ones_like(ops[3]))
    ref, _ = _reference(*ops, sizes, starts)
    routed = ~np.isnan(ref)
    want = ref[routed] if c_type == mg.TYPE_F32 else nu.round_bf16(ref[routed])
    ops = padded(ops)
    for workspace in (True, False):
        c = _product(*ops, sizes, starts, c_type, workspace=workspace, **kw)
        got = c[:starts[-1]].double().cpu().numpy()
        np.testing.assert_array_equal(got[routed], want)
        assert (got[~routed] == -77.0).all() and bool((c[starts[-1]:] == -77.0).all())
    ops = _operands(rng, sizes, starts, starts[-1], N, K)
    ref, mag = _reference(*ops, sizes, starts)
    ops = padded(ops)
    c = _product(*ops, sizes, starts, c_type, **kw)
    _check(c[:starts[-1]], ref, mag, K, c_type == mg.TYPE_BF16)
    assert torch.equal(c, _product(*ops, sizes, starts, c_type, **kw))
    # the order moves an fp32 sum by some 2^-23, and one bf16 output of 10^4 past the
    # border of two: of 41 x 272 that may be none, of 379 x 272 and more it is ten
    if c_type == mg.TYPE_F32 or sum(sizes) > 300:
        assert not torch.equal(c, _product(*ops, sizes, starts, c_type, workspace=False, **kw))


def test_pad_rows_of_the_layer_encode_zeros():
    """The weight gradient reads the pad rows of a group's last block: the
    codes that the layer stores there are zeros, also after a step that filled
    them, and the gradient is that of the routed rows alone."""
    E, k, T, H, I = 6, 2, 150, 128, 192
    blk = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8, wgrad=True, wgrad_type=mg.TYPE_F32)
    x, dout, w1, w2, _ = _inputs(E, H, 2 * I, I, T, 3)
    blk.load_weights(w1, w2)
    probs = torch.full((T, k), 0.5, device=DEV)
    for seed in range(3):
        idx = torch.rand(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)).topk(k, dim=1).indices.to(torch.int32)
        if seed == 2:
            idx[:] = torch.tensor([1, 4], dtype=torch.int32)
        blk.forward(x, idx, probs)
        blk.backward(dout)
        blk.weight_grads()
        torch.cuda.synchronize()
        sizes, starts = blk.split_sizes.tolist(), blk.padded_offsets.tolist()
        pads = np.ones(starts[-1], bool)
        for n, o in zip(sizes, starts):
            pads[o:o + n] = False
        assert pads.any()
        for left, right, dw in (("dz", "xp", blk.dw1), ("dyp", "a", blk.dw2)):
            ops = []
            for n in (left, right):
                q = getattr(blk, n + "T_q8").cpu().numpy()[:, :starts[-1]]
                assert (q[:, pads] & 0x7F == 0).all(), n
                v = st.dequantize_rows(q, getattr(blk, n + "T_s8").cpu().numpy()[:starts[-1] // 128])
                ops.append(np.where(pads[None, :], 0.0, v))
            ref, mag = st.grouped_weight_grad(*ops, sizes, starts)
            tol = 2 * (128 + starts[-1] // 128 + 4) * 2.0 ** -23 * mag
            assert (np.abs(dw.double().cpu().numpy() - ref) <= tol).all()
