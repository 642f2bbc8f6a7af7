"""ExpertBlock with the router by scores, the AdamW step and the 8-bit integer
layer, run together as a training step and as a serving step.

Each stage is held to the oracle on the operands the GPU itself stored.
Tolerances: integer products bit for bit; the activation against float64 with
its own two roundings (fp32 evaluation, 2^-16 of it for the fast exponential and
reciprocal, then bf16, 2^-8); weights after a step as in test_gpu_adamw."""

import gc

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import layer as ol

from .test_gpu_adamw import U
from .test_gpu_fp8_block import _host, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """Tests after these measure what torch's allocator holds."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


DEV = "cuda"
GATE = dict(score=mg.SCORE_SIGMOID, n_groups=4, topk_groups=2, group_top=2, renorm=True, scale=2.5)
ORACLE_GATE = dict(sigmoid=True, n_groups=4, topk_groups=2, group_top=2, renorm=True, scale=2.5)


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _product(blk, name, weight, c, rows):
    sizes, starts = blk.split_sizes.tolist(), blk.padded_offsets.tolist()
    ref = ol.product_int8(*(getattr(blk, n).cpu().numpy() for n in (name + "_qi", name + "_si", weight + "_qi", weight + "_si")),
                          sizes, starts, blk.M_cap)[:rows]
    inside = ~np.isnan(ref)
    want = torch.from_numpy(ref).to(torch.bfloat16)
    assert torch.equal(c[:rows].cpu()[torch.from_numpy(inside)], want[torch.from_numpy(inside)])


@pytest.mark.parametrize("T,k,E,H,I", [(64, 4, 16, 256, 128), (5, 2, 8, 288, 192), (300, 8, 16, 512, 320), (1, 1, 4, 128, 64)])
def test_serving_layer(T, k, E, H, I):
    groups = 4
    x, _, w1, w2, logits = _inputs(E, H, 2 * I, I, T, T)
    blk = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_INT8)
    blk.load_weights(w1, w2)
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    if T > 4:
        mask[2] = False   # a token of the padding
    stay = 2 if k <= 2 * E // groups else groups
    kw = {**GATE, "topk_groups": stay}
    blk.gate(logits, x, token_mask=mask, **kw)
    idx, w = ol.gate(_host(logits), k, mask=mask.cpu().numpy(), **{**ORACLE_GATE, "topk_groups": stay})
    np.testing.assert_array_equal(blk.expert_idx.cpu().numpy(), idx)
    out = blk.forward(x, blk.expert_idx, blk.probs)
    rows = int(blk.padded_offsets[-1])
    for name, weights in (("w1", blk.w1i), ("w2", blk.w2)):
        q, s = ol.quantize_int8(_host(weights).reshape(-1, weights.shape[-1]))
        np.testing.assert_array_equal(getattr(blk, name + "_qi").cpu().numpy().reshape(q.shape), q)
        np.testing.assert_array_equal(getattr(blk, name + "_si").cpu().numpy().reshape(-1), s)
    for name, src, weight, dst in (("xp", blk.xp, "w1", blk.z), ("a", blk.a, "w2", blk.yp)):
        q, s = ol.quantize_int8(_host(src)[:rows])
        np.testing.assert_array_equal(getattr(blk, name + "_qi").cpu().numpy()[:rows], q)
        np.testing.assert_array_equal(getattr(blk, name + "_si").cpu().numpy()[:rows], s)
        _product(blk, name, weight, dst, rows)
    # the combine: each token's rows in the order of its slots, in fp32
    yp, rid = _host(blk.yp), blk.row_id_map.cpu().numpy()
    ref = np.stack([sum((yp[r] for r in rid[t] if r >= 0), np.zeros(H)) for t in range(T)])
    mag = np.stack([sum((np.abs(yp[r]) for r in rid[t] if r >= 0), np.zeros(H)) for t in range(T)])
    assert (np.abs(_host(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 16 * U * mag).all()
    if T > 4:
        assert not out[2].any() and (rid[2] == -1).all()
    assert blk.err_flag.item() == 0
    # against the layer in float64 with no rounding at all: each of the two 8-bit
    # roundings of a product is off by half a code of the row's largest value
    z = np.zeros((T, H))
    w1n, w2n, xn = _host(w1), _host(w2), _host(x)
    for t in range(T):
        for j in range(k):
            if idx[t, j] >= 0:
                g, u = np.split(w1n[idx[t, j]] @ xn[t], 2)
                z[t] += w2n[idx[t, j]] @ (w[t, j] * g / (1 + np.exp(-g)) * u)
    if z.any():
        assert np.linalg.norm(_host(out) - z) <= 0.05 * np.linalg.norm(z)


def test_serving_layer_has_no_backward():
    blk = mg.ExpertBlock(2, 128, 64, 4, 1, prec=mg.PREC_INT8)
    with pytest.raises(RuntimeError):
        blk.backward(torch.zeros(4, 128, dtype=torch.bfloat16, device=DEV))
    for kw in (dict(wgrad=True), dict(recompute=True), dict(unfused=True)):
        with pytest.raises(ValueError):
            mg.ExpertBlock(2, 128, 64, 4, 1, prec=mg.PREC_INT8, **kw)


def _step(blk, x, dout, logits, bias, lr, **kw):
    blk.gate(logits, x, bias=bias, count=True, **GATE)
    blk.forward(x, blk.expert_idx, blk.probs)
    blk.backward(dout)
    dlogits = blk.gate_backward()
    blk.weight_grads()
    blk.adamw_step(lr, weight_decay=0.1, max_norm=0.5, **kw)
    blk.update_bias(bias, 0.01)
    return dlogits


@pytest.mark.parametrize("prec", [mg.PREC_BF16, mg.PREC_FP8])
@pytest.mark.parametrize("state,master", [(mg.STATE_F32, True), (mg.STATE_FP8, False)])
def test_training_steps(prec, state, master):
    E, k, T, H, I = 16, 4, 200, 128, 128
    x, dout, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 3)
    blk = mg.ExpertBlock(E, H, I, T, k, prec=prec, wgrad=True)
    blk.load_weights(w1, w2)
    bias = torch.zeros(E, device=DEV)
    own = [_host(blk.w1i).ravel(), _host(blk.w2).ravel()]
    ms, vs = [np.zeros_like(w) for w in own], [np.zeros_like(w) for w in own]
    for step in (1, 2, 3):
        before = bias.clone()
        dlogits = _step(blk, x, dout, logits, bias, 1e-2, state=state, master=master, stochastic=state == mg.STATE_FP8, seed=step)
        idx, _ = ol.gate(_host(logits), k, bias=_host(before), **ORACLE_GATE)
        np.testing.assert_array_equal(blk.expert_idx.cpu().numpy(), idx)
        np.testing.assert_array_equal(bias.cpu().numpy(), ol.bias_update(np.bincount(idx.ravel(), minlength=E), before.cpu().numpy(), 0.01))
        assert not blk.gate_counts.any()
        ref, mag = ol.gate_bwd(_host(logits), idx, _host(blk.dprobs), True, True, 2.5)
        assert (np.abs(_host(dlogits) - ref) <= 60 * 2.0 ** -23 * mag + 1e-40).all()
        grads = [_host(blk.dw1).ravel(), _host(blk.dw2).ravel()]
        f = ol.clip_factor(sum((g * g).sum() for g in grads), 0.5)
        for i, (w, g) in enumerate(zip((blk.w1i, blk.w2), grads)):
            w1_, m1, v1, gm, den = ol.adamw(own[i], g, ms[i], vs[i], 1e-2, 0.9, 0.999, 1e-8, 0.1, step, f)
            upd = 1e-2 / (1 - 0.9 ** step) / den
            # (squares of the smallest gradients leave fp32's normal range)
            tol = upd * 6 * U * gm + 30 * U * upd * np.abs(m1) + 3 * U * np.abs(own[i]) + upd * np.abs(m1) * (v1 < 2.0 ** -110) + 2.0 ** -149
            final = tol + 2.0 ** -8 * (np.abs(w1_) + tol)
            assert (np.abs(_host(w).ravel() - w1_) <= final).all(), (step, i)
            # go on from what the block holds
            own[i] = _host(blk._adamw["master"][i]) if master else _host(w).ravel()
            if state == mg.STATE_F32:
                ms[i], vs[i] = _host(blk._adamw["m"][i]), _host(blk._adamw["v"][i])
            else:
                n = len(own[i])
                ms[i] = _host(blk._adamw["m"][i].view(torch.float8_e4m3fn)) * ol.spread(_host(blk._adamw["m_scale"][i]), n)
                vs[i] = (_host(blk._adamw["v"][i].view(torch.float8_e4m3fn)) * ol.spread(_host(blk._adamw["v_scale"][i]), n)) ** 2
        if prec == mg.PREC_FP8:   # the products' copies are of the new weights
            q, s = blk.w2_q8.clone(), blk.w2_s8.clone()
            blk.quantize_weights()
            assert torch.equal(q, blk.w2_q8) and torch.equal(s, blk.w2_s8)
    assert blk.err_flag.item() == 0


def test_captured_training_steps():
    """A whole step in a graph, replayed: the same as eager steps, bit for bit."""
    E, k, T, H, I = 8, 2, 100, 128, 128
    x, dout, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 4)
    blocks, biases = [], []
    for _ in range(2):
        blk = mg.ExpertBlock(E, H, I, T, k, wgrad=True)
        blk.load_weights(w1, w2)
        blocks.append(blk)
        biases.append(torch.zeros(E, device=DEV))
    lr = torch.full((1,), 1e-2, device=DEV)
    for blk, bias in zip(blocks, biases):   # the first step makes states and buffers
        _step(blk, x, dout, logits, bias, lr, capturable=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(blocks[0], x, dout, logits, biases[0], lr, capturable=True)
    for step in range(4):
        lr.fill_(1e-2 / (step + 1))
        graph.replay()
        _step(blocks[1], x, dout, logits, biases[1], lr, capturable=True)
        torch.cuda.synchronize()
        for a, b in ((blocks[0].w1i, blocks[1].w1i), (blocks[0].w2, blocks[1].w2), tuple(biases), (blocks[0]._adamw["step"], blocks[1]._adamw["step"]),
                     (blocks[0]._adamw["v"][1], blocks[1]._adamw["v"][1]), (blocks[0].expert_idx, blocks[1].expert_idx)):
            assert torch.equal(a, b)
    assert blocks[0]._adamw["step"].item() == 5   # the eager one and four replays


def test_gate_adds_to_the_losses_gradient():
    E, k, T, H, I = 16, 4, 64, 128, 64
    x, dout, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 5)
    blk = mg.ExpertBlock(E, H, I, T, k)
    blk.load_weights(w1, w2)
    blk.gate(logits, renorm=True)
    blk.forward(x, blk.expert_idx, blk.probs)
    blk.backward(dout)
    alone = blk.gate_backward().clone()
    blk.router_loss(logits, balance_coef=0.1, z_coef=0.01)
    losses = blk.router_backward(dprobs=torch.zeros(T, k, device=DEV)).clone()
    both = blk.gate_backward(dlogits=losses.clone(), accumulate=True)
    assert torch.allclose(both, alone + losses, rtol=1e-6, atol=1e-7 * float(alone.abs().max()))


def test_refusals():
    blk = mg.ExpertBlock(8, 128, 64, 16, 2, wgrad=True)
    logits = torch.zeros(16, 8, device=DEV)
    with pytest.raises(RuntimeError):
        blk.gate_backward()
    with pytest.raises(RuntimeError):
        blk.update_bias(torch.zeros(8, device=DEV), 0.1)
    with pytest.raises(ValueError):
        blk.gate(torch.zeros(15, 8, device=DEV))
    blk.gate(logits)
    with pytest.raises(RuntimeError):
        blk.gate_backward()   # no backward() yet
    for bad in (dict(dprobs=torch.zeros(15, 2, device=DEV)), dict(dprobs=torch.zeros(16, 2, device=DEV), accumulate=True),
                dict(dprobs=torch.zeros(16, 2, device=DEV), dlogits=torch.zeros(16, 7, device=DEV)),
                dict(dprobs=torch.zeros(16, 2, device=DEV), dlogits=logits.bfloat16())):
        with pytest.raises(ValueError):
            blk.gate_backward(**bad)
    blk.dw1.zero_()
    blk.dw2.zero_()
    blk.w1i.zero_()
    blk.w2.zero_()
    with pytest.raises(RuntimeError):
        blk.adamw_step(torch.ones(1, device=DEV))
    blk.adamw_step(0.1)
    with pytest.raises(ValueError):
        blk.adamw_step(0.1, state=mg.STATE_FP8)
    with pytest.raises(RuntimeError):
        mg.ExpertBlock(8, 128, 64, 16, 2).adamw_step(0.1)


def test_shards_of_the_experts_add_up():
    """Two blocks with half of the experts each, fed the same logits; every output
    is off by one rounding, and the sums by fp32's."""
    E, k, T, H, I = 16, 4, 50, 256, 128
    x, _, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 8)
    outs, mags = [], []
    for first, n in ((0, E), (0, E // 2), (E // 2, E // 2)):
        blk = mg.ExpertBlock(n, H, I, T, k, prec=mg.PREC_INT8, first_expert=first)
        blk.load_weights(w1[first:first + n].contiguous(), w2[first:first + n].contiguous())
        blk.gate(logits, count=True, **GATE)
        outs.append(_host(blk.forward(x, blk.expert_idx, blk.probs)))
        yp, rid = _host(blk.yp), blk.row_id_map.cpu().numpy()
        mags.append(np.stack([sum((np.abs(yp[r]) for r in rid[t] if r >= 0), np.zeros(H)) for t in range(T)]))
        assert int(blk.gate_counts.sum()) == T * k and blk.err_flag.item() == 0   # (of all experts)
    tol = 2.0 ** -8 * sum(np.abs(o) + 16 * U * m for o, m in zip(outs, mags)) + 16 * U * sum(mags)
    assert np.abs(outs[0]).max() > 0 and (np.abs(outs[0] - outs[1] - outs[2]) <= tol).all()


def test_captured_serving_step():
    """Router and layer in a graph, replayed with other tokens: as eager calls."""
    E, k, T, H, I = 8, 2, 6, 256, 128
    x, _, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 9)
    blocks = [mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_INT8) for _ in range(2)]
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)

    def step(blk):
        blk.gate(logits, token_mask=mask, count=True, **GATE)
        return blk.forward(x, blk.expert_idx, blk.probs)

    for blk in blocks:
        blk.load_weights(w1, w2)
        step(blk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(blocks[0])
    for i in range(4):
        x.copy_(torch.randn(T, H, device=DEV))
        logits.copy_(torch.randn(T, E, device=DEV))
        mask.fill_(1)
        mask[i:i + 2] = 0
        graph.replay()
        want = step(blocks[1])
        torch.cuda.synchronize()
        assert torch.equal(out, want) and not out[i:i + 2].any() and out[(i + 3) % T].any()
        assert torch.equal(blocks[0].gate_counts, blocks[1].gate_counts)


def test_two_layers_on_two_streams_at_once():
    """Nothing is shared between calls: layers that run side by side give what
    each gives alone."""
    E, k, T, H, I = 8, 2, 700, 512, 512
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets, alone = [], []
    for seed in (10, 11):
        x, _, w1, w2, logits = _inputs(E, H, 2 * I, I, T, seed)
        blk = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_INT8)
        blk.load_weights(w1, w2)
        sets.append((blk, x, logits))
        blk.gate(logits, **GATE)
        alone.append(blk.forward(x, blk.expert_idx, blk.probs).clone())
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, (blk, x, logits) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                blk.gate(logits, **GATE)
                got[i] = blk.forward(x, blk.expert_idx, blk.probs)
    torch.cuda.synchronize()
    for a, b in zip(got, alone):
        assert torch.equal(a, b)
