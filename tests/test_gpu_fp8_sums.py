"""How the block-scaled FP8 products sum: in fp32, whatever the output's type.

Within every other group of eight neighbours along the contraction axis two
large products (448 * 64) cancel, and the rest are integers of at most 49.
Every partial sum in any order is an integer below 2^24, so fp32 sums are
exact and the outputs are the oracle's to the bit; sums that keep 13 bits
below the largest of eight products would lose the small ones."""

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import numerics as nu
from oracle import step as st

from .test_gpu_fp8 import (HINTS, SHAPES, SIZES, WSIZES, _check, _margin, _operands, _product, _reference, _starts, _wgrad,
                           _wgrad_operands, _wgrad_ref)
from .test_gpu_fp8_block import _inputs

pytestmark = pytest.mark.gpu


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _cancelling(a_q, b_q, used):
    """Large products that cancel, in columns k and k + 1 of every 16 (both of
    them used, or neither gets any)."""
    a, b = a_q.copy(), b_q.copy()
    big, neg, w = (nu.e4m3_encode(np.array([v]))[0] for v in (448.0, -448.0, 64.0))
    for k in range(0, a.shape[-1] - 1, 16):
        if used[k] and used[k + 1]:
            a[..., k], a[..., k + 1] = big, neg
            b[..., k] = b[..., k + 1] = w
    return a, b


@pytest.mark.parametrize("c_type", [mg.TYPE_F32, mg.TYPE_BF16])
@pytest.mark.parametrize("hint", HINTS)
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("name", SIZES)
def test_product_sums_in_fp32(name, N, K, hint, c_type):
    sizes = SIZES[name]
    rng = np.random.default_rng(N + K + len(name))
    starts = _starts(sizes)
    a_q, a_s, b_q, b_s = _operands(rng, sizes, starts, max(128, starts[-1]), N, K, exact=True)
    nan = a_q == 0x7F
    a_q, b_q = _cancelling(a_q, b_q, np.ones(K, bool))
    a_q[nan] = 0x7F
    ref, _ = _reference(a_q, a_s, b_q, b_s, sizes, starts)
    c = _product(a_q, a_s, b_q, b_s, sizes, starts, c_type, hint).double().cpu().numpy()
    routed = ~np.isnan(ref)
    want = ref if c_type == mg.TYPE_F32 else nu.round_bf16(ref)
    np.testing.assert_array_equal(c[routed], want[routed])
    assert (c[~routed] == -77.0).all()


@pytest.mark.parametrize("leave", [1, 9, 40])
@pytest.mark.parametrize("c_type", [mg.TYPE_F32, mg.TYPE_BF16])
@pytest.mark.parametrize("name", WSIZES)
def test_wgrad_sums_in_fp32(name, c_type, leave):
    sizes, P, Q = WSIZES[name], 272, 528
    starts = _starts(sizes)
    rng = np.random.default_rng(len(name))
    a_q, a_s, b_q, b_s = _wgrad_operands(rng, sizes, starts, max(256, starts[-1] + 128), P, Q, exact=True)
    used = np.zeros(a_q.shape[1], bool)
    for n, o in zip(sizes, starts):
        used[o:o + n] = True
    a_q, b_q = _cancelling(a_q, b_q, used)
    ref, _ = _wgrad_ref(a_q, a_s, b_q, b_s, sizes, starts)
    c = _wgrad(a_q, a_s, b_q, b_s, sizes, starts, c_type, cu_margin=_margin(leave)).double().cpu().numpy()
    np.testing.assert_array_equal(c, ref if c_type == mg.TYPE_F32 else nu.round_bf16(ref))


# ------------------------------------- fp8_sums: the sums inside a block ---
# Small integers, whose products the FP8 instructions add exactly, and random
# data within their bound.
@pytest.mark.parametrize("leave", [0, 1, 9, 20])
@pytest.mark.parametrize("hint", [16, 32, 0])
@pytest.mark.parametrize("name", SIZES)
def test_product_by_fp8_sums(name, hint, leave):
    sizes, N, K = SIZES[name], 272, 400
    rng = np.random.default_rng(leave)
    starts = _starts(sizes)
    kw = dict(max_rows=hint, fp8_sums=True, cu_margin=_margin(leave) if leave else 0)
    ops = _operands(rng, sizes, starts, max(128, starts[-1]), N, K, exact=True)
    ref, _ = _reference(*ops, sizes, starts)
    c = _product(*ops, sizes, starts, mg.TYPE_BF16, **kw).double().cpu().numpy()
    np.testing.assert_array_equal(c[~np.isnan(ref)], nu.round_bf16(ref[~np.isnan(ref)]))
    assert (c[np.isnan(ref)] == -77.0).all()
    ops = _operands(rng, sizes, starts, max(128, starts[-1]), N, K)
    ref, mag = _reference(*ops, sizes, starts)
    _check(_product(*ops, sizes, starts, mg.TYPE_BF16, **kw), ref, mag, K, True)


@pytest.mark.parametrize("leave", [1, 20, 40, 80])
@pytest.mark.parametrize("name", WSIZES)
def test_wgrad_by_fp8_sums(name, leave):
    sizes, P, Q = WSIZES[name], 592, 272
    starts = _starts(sizes)
    rng = np.random.default_rng(leave)
    M_cap = max(256, starts[-1] + 128)
    kw = dict(fp8_sums=True, cu_margin=_margin(leave))
    ops = _wgrad_operands(rng, sizes, starts, M_cap, P, Q, exact=True)
    ref, _ = _wgrad_ref(*ops, sizes, starts)
    np.testing.assert_array_equal(_wgrad(*ops, sizes, starts, mg.TYPE_BF16, **kw).double().cpu().numpy(), nu.round_bf16(ref))
    ops = _wgrad_operands(rng, sizes, starts, M_cap, P, Q)
    ref, mag = _wgrad_ref(*ops, sizes, starts)
    c = _wgrad(*ops, sizes, starts, mg.TYPE_BF16, **kw).double().cpu().numpy()
    # (as test_wgrad_random has it)
    tol = (2 * (128 + M_cap // 128 + 4) * 2.0 ** -23 + 7 * 2.0 ** -13) * mag
    assert (np.abs(c - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol)).all()


def test_fp8_sums_cut_along_k():
    sizes, N, K = [33, 0, 260, 1], 272, 3152
    starts = _starts(sizes)
    ops = _operands(np.random.default_rng(3), sizes, starts, starts[-1], N, K)
    ref, mag = _reference(*ops, sizes, starts)
    c = _product(*ops, sizes, starts, mg.TYPE_BF16, fp8_sums=True)
    _check(c, ref, mag, K, True)
    assert torch.equal(c, _product(*ops, sizes, starts, mg.TYPE_BF16, fp8_sums=True))
    assert not torch.equal(c, _product(*ops, sizes, starts, mg.TYPE_BF16, fp8_sums=True, workspace=False))
    assert not torch.equal(c, _product(*ops, sizes, starts, mg.TYPE_BF16))


@pytest.mark.parametrize("wtype", [mg.TYPE_BF16, mg.TYPE_F32])
def test_layer_passes_fp8_sums_on(wtype):
    """The layer's products are the calls' with the same switch."""
    E, k, T, H, I = 4, 2, 200, 256, 320
    x, dout, w1, w2, logits = _inputs(E, H, 2 * I, I, T, 1)
    outs = []
    for fast in (False, True):
        blk = mg.ExpertBlock(E, H, I, T, k, prec=mg.PREC_FP8, wgrad=True, wgrad_type=wtype, fp8_sums=fast)
        blk.load_weights(w1, w2)
        blk.route_logits(logits)
        blk.forward(x, blk.expert_idx, blk.probs)
        blk.backward(dout)
        dw1, _ = blk.weight_grads()
        rows = blk.padded_offsets[-1].item()
        size = dict(E=E, M_cap=blk.M_cap, split_sizes=blk.split_sizes, padded_offsets=blk.padded_offsets)
        z, c = torch.zeros_like(blk.z), torch.zeros_like(dw1)
        mg.moe_grouped_gemm_fp8(**size, N=2 * I, K=H, a=blk.xp_q8, a_s=blk.xp_s8, b=blk.w1_q8, b_s=blk.w1_s8, c=z, fp8_sums=fast,
                                max_rows=T, workspace=blk.ws)
        mg.moe_grouped_wgrad_fp8(**size, P=2 * I, Q=H, a=blk.dzT_q8, a_s=blk.dzT_s8, b=blk.xpT_q8, b_s=blk.xpT_s8, c=c,
                                 c_type=wtype, fp8_sums=fast and wtype == mg.TYPE_BF16)
        for n, o in zip(blk.split_sizes.tolist(), blk.padded_offsets.tolist()):
            assert torch.equal(z[o:o + n], blk.z[o:o + n])
        assert torch.equal(c, dw1)
        outs.append(blk.out.clone())
    assert not torch.equal(*outs) and rows


# --------------------------------------------------- NaN and infinite blocks ---
VARIANTS = [dict(c_type=mg.TYPE_F32), dict(c_type=mg.TYPE_BF16), dict(c_type=mg.TYPE_BF16, fp8_sums=True)]


@pytest.mark.parametrize("kw", VARIANTS)
@pytest.mark.parametrize("hint", [16, 32, 0])
@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_product_nan_and_infinite_blocks(code, hint, kw):
    """A NaN code makes its token's row NaN, or its weight row's column of the
    expert; a block whose scale is infinite (codes zero but for a NaN, as the
    quantizer writes it) makes the row NaN; all else is as without them."""
    sizes, N, K = [3, 0, 40, 17], 144, 400
    starts = _starts(sizes)
    a_q, a_s, b_q, b_s = _operands(np.random.default_rng(7), sizes, starts, starts[-1], N, K, exact=True)
    clean = _product(a_q, a_s, b_q, b_s, sizes, starts, max_rows=hint, **kw).double().cpu().numpy()
    r0, r1 = starts[2] + 5, starts[3] + 16
    a_q[r0, 399] = code
    a_q[r1, 128:256] = 0
    a_q[r1, 200] = code
    a_s[1, r1] = np.inf
    b_q[2, 77, 130] = code
    c = _product(a_q, a_s, b_q, b_s, sizes, starts, max_rows=hint, **kw).double().cpu().numpy()
    bad = np.zeros(c.shape, bool)
    bad[[r0, r1]] = True
    bad[starts[2]:starts[2] + sizes[2], 77] = True
    np.testing.assert_array_equal(np.isnan(c), bad)
    np.testing.assert_array_equal(c[~bad], clean[~bad])


@pytest.mark.parametrize("kw", VARIANTS)
def test_wgrad_nan_and_infinite_blocks(kw):
    sizes, P, Q = [130, 0, 3], 80, 272
    starts = _starts(sizes)
    a_q, a_s, b_q, b_s = _wgrad_operands(np.random.default_rng(8), sizes, starts, starts[-1], P, Q, exact=True)
    clean = _wgrad(a_q, a_s, b_q, b_s, sizes, starts, **kw).double().cpu().numpy()
    a_q[5, 129] = 0x7F                       # expert 0, second block
    b_q[260, starts[2]:starts[2] + 3] = [0, 0xFF, 0]   # expert 2
    b_s[starts[2] // 128, 260] = np.inf
    c = _wgrad(a_q, a_s, b_q, b_s, sizes, starts, **kw).double().cpu().numpy()
    bad = np.zeros(c.shape, bool)
    bad[0, 5] = True
    bad[2, :, 260] = True
    np.testing.assert_array_equal(np.isnan(c), bad)
    np.testing.assert_array_equal(c[~bad], clean[~bad])
