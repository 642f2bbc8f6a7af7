"""Host-side checks of the block-scaled FP8, router-loss and gradient entry
points (no GPU needed): struct layout, refusals before a device is touched,
workspace sizes, and the binding's own tensor checks.

The C calls pass placeholder addresses, so the ones that would be valid run
only where no HIP device is present."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import moe_grouped_mlp_amd as m
from moe_grouped_mlp_amd import binding as B

from .test_abi import DEVICE, HEADER, INVALID, UNSUPPORTED, WORKSPACE, _call, no_device

NAN, INF = float("nan"), float("inf")

STRUCTS = {
    "moe_quant_fp8_args": B.QuantFp8Args,
    "moe_gemm_fp8_args": B.GemmFp8Args,
    "moe_wgrad_fp8_args": B.WgradFp8Args,
    "moe_router_loss_args": B.RouterLossArgs,
    "moe_router_bwd_args": B.RouterBwdArgs,
    "moe_tensor": B.Tensor,
    "moe_grad_args": B.GradArgs,
}


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc missing")
def test_ctypes_structs_match_header_layout(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void) {"]
    for cname, st in STRUCTS.items():
        lines.append(f'printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in st._fields_]
    lines += ["return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c11", "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out if line}
    for cname, st in STRUCTS.items():
        assert got[(cname, "sizeof")] == ctypes.sizeof(st), cname
        for f, _ in st._fields_:
            assert got[(cname, f)] == getattr(st, f).offset, (cname, f)


def test_constants():
    text = open(HEADER).read()
    assert f"#define MOE_FP8_BLOCK {m.FP8_BLOCK}" in text
    assert f"#define MOE_QUANT_TILE {m.QUANT_TILE}" in text
    assert f"#define MOE_DEVERR_NONFINITE 0x{m.DEVERR_NONFINITE:x}" in text
    assert f"MOE_TYPE_BF16 = {m.TYPE_BF16}, MOE_TYPE_F32 = {m.TYPE_F32}" in text


def _make(st, base):
    def make(**kw):
        a = st()
        for k, v in {**base, **kw}.items():
            setattr(a, k, v)
        return a
    return make


def _refuses(fn, make, cases, status=INVALID):
    for kw in cases:
        assert _call(fn, make(**kw)) == status, (fn, kw)


quant = _make(B.QuantFp8Args, dict(mode=m.QUANT_BOTH, batch=2, rows=32, cols=48, x=64, q=64, s=64, qT=64, sT=64))
gemm = _make(B.GemmFp8Args, dict(E=4, N=48, K=144, M_cap=512, split_sizes=64, padded_offsets=64, a=64, a_s=64, b=64, b_s=64, c=64))
wgrad = _make(B.WgradFp8Args, dict(E=4, P=48, Q=144, M_cap=512, split_sizes=64, padded_offsets=64, a=64, a_s=64, b=64, b_s=64, c=64))
loss = _make(B.RouterLossArgs, dict(T=16, E=8, k=2, logits=64, expert_idx=64, counts=64, n_tokens=64, prob_mean=64, loss=64,
                                    workspace=64, workspace_bytes=1 << 20, balance_coef=0.1, z_coef=0.1))
bwd = _make(B.RouterBwdArgs, dict(T=16, E=8, k=2, logits=64, expert_idx=64, counts=64, n_tokens=64, dlogits=64, balance_coef=0.1, z_coef=0.1))


def test_null_arguments():
    for fn in ("moe_quantize_fp8", "moe_grouped_gemm_fp8", "moe_grouped_wgrad_fp8", "moe_router_loss", "moe_router_bwd",
               "moe_grad_sumsq", "moe_grad_clip"):
        assert getattr(m.lib(), fn)(None, None) == INVALID


def test_quantize_refusals():
    _refuses("moe_quantize_fp8", quant, [
        dict(mode=-1), dict(mode=4), dict(batch=-1), dict(rows=-16), dict(rows=24), dict(cols=0), dict(cols=40), dict(cols=-16),
        dict(x=None), dict(q=None), dict(s=None), dict(qT=None), dict(sT=None), dict(x=8), dict(q=4), dict(qT=8),
        dict(x_stride=100), dict(x_stride=32 * 48 + 4), dict(mode=m.QUANT_TILE, sT=None), dict(mode=m.QUANT_TILE, qT=None)])
    _refuses("moe_quantize_fp8", quant, [dict(batch=65536), dict(mode=m.QUANT_TILE, rows=1 << 30, cols=1 << 20)], UNSUPPORTED)


@no_device
def test_quantize_accepts():
    _refuses("moe_quantize_fp8", quant, [
        dict(), dict(mode=m.QUANT_ROW, rows=7, qT=None, sT=None), dict(mode=m.QUANT_TILE, qT=None, sT=None),
        dict(x_stride=32 * 48 + 8), dict(rows=0), dict(batch=0), dict(mode=m.QUANT_COL, qT=None, sT=None)], DEVICE)


def test_product_refusals():
    _refuses("moe_grouped_gemm_fp8", gemm, [
        dict(E=0), dict(E=1025), dict(N=0), dict(N=40), dict(K=0), dict(K=100), dict(K=(1 << 22) + 16), dict(M_cap=0),
        dict(M_cap=1 << 31), dict(split_sizes=None), dict(padded_offsets=None), dict(a=None), dict(a_s=None), dict(b=None),
        dict(b_s=None), dict(c=None), dict(a=72), dict(b=72), dict(c=72), dict(c_type=2), dict(c_type=-1), dict(max_rows=-1),
        dict(cu_margin=-1), dict(b_stride=48), dict(b_stride=48 * 144 + 8), dict(b_s_stride=1), dict(ldc=40), dict(ldc=52)])
    _refuses("moe_grouped_gemm_fp8", gemm, [dict(M_cap=(1 << 31) - 1, N=1 << 30)], UNSUPPORTED)


@no_device
def test_product_accepts():
    _refuses("moe_grouped_gemm_fp8", gemm, [
        dict(), dict(c_type=1), dict(max_rows=1), dict(ldc=56), dict(b_stride=48 * 144 + 16, b_s_stride=3), dict(M_cap=1)], DEVICE)


def test_wgrad_refusals():
    _refuses("moe_grouped_wgrad_fp8", wgrad, [
        dict(E=0), dict(E=1025), dict(P=0), dict(P=40), dict(Q=8), dict(Q=-16), dict(M_cap=0), dict(M_cap=500),
        dict(M_cap=4194304 + 128), dict(split_sizes=None), dict(padded_offsets=None), dict(a=None), dict(a_s=None),
        dict(b=None), dict(b_s=None), dict(c=None), dict(a=72), dict(b=72), dict(c=72), dict(c_type=3), dict(accumulate=1),
        dict(cu_margin=-1)])


@no_device
def test_wgrad_accepts():
    _refuses("moe_grouped_wgrad_fp8", wgrad, [dict(), dict(c_type=1, accumulate=1)], DEVICE)


def test_router_loss_refusals():
    _refuses("moe_router_loss", loss, [
        dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=4, k=5), dict(T=1 << 30, k=8, E=8), dict(logits=None),
        dict(expert_idx=None), dict(counts=None), dict(n_tokens=None), dict(prob_mean=None), dict(loss=None),
        dict(balance_coef=NAN), dict(balance_coef=INF), dict(z_coef=NAN), dict(z_coef=-INF)])
    _refuses("moe_router_loss", loss, [dict(workspace=None), dict(workspace_bytes=8), dict(workspace=66)], WORKSPACE)


def test_router_bwd_refusals():
    _refuses("moe_router_bwd", bwd, [
        dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(logits=None), dict(expert_idx=None), dict(dlogits=None),
        dict(counts=None), dict(n_tokens=None), dict(balance_coef=0.0, n_tokens=None), dict(balance_coef=NAN), dict(z_coef=INF)])


@no_device
def test_router_accepts():
    _refuses("moe_router_loss", loss, [dict(), dict(T=0, logits=None, expert_idx=None), dict(token_mask=64)], DEVICE)
    _refuses("moe_router_bwd", bwd, [
        dict(), dict(T=0, logits=None, expert_idx=None, dlogits=None),
        dict(counts=None, n_tokens=None, balance_coef=0.0, z_coef=0.0, dprobs=64)], DEVICE)


def _list(*tensors):
    arr = (B.Tensor * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        arr[i] = B.Tensor(*t)
    return arr


def _grad(tensors, n=None, **kw):
    a = B.GradArgs(_list(*tensors), len(tensors) if n is None else n, 1.0, 64, None, None, 64, 1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_TENSORS = [(None, None, 4, 0), (64, None, -1, 0), (64, None, 4, 2), (64, None, 4, -1), (65, None, 4, 0), (66, None, 4, 1),
               (64, 130, 4, 1), (64, None, 1 << 47, 0)]


@pytest.mark.parametrize("fn", ["moe_grad_sumsq", "moe_grad_clip"])
def test_grad_refusals(fn):
    ok = (64, None, 4, 1)
    for bad in BAD_TENSORS:
        assert _call(fn, _grad([ok, bad])) == INVALID, bad
    assert _call(fn, _grad([ok], n=-1)) == INVALID
    assert _call(fn, _grad([ok], sumsq=None)) == INVALID
    assert _call(fn, _grad([ok], sumsq=68)) == INVALID
    a = _grad([ok])
    a.tensors = ctypes.POINTER(B.Tensor)()
    assert _call(fn, a) == INVALID
    if fn == "moe_grad_sumsq":
        assert _call(fn, _grad([ok], workspace=None)) == WORKSPACE
        assert _call(fn, _grad([ok], workspace_bytes=100)) == WORKSPACE
        assert _call(fn, _grad([ok], workspace=68)) == WORKSPACE
    else:
        for v in (-1.0, NAN):
            assert _call(fn, _grad([ok], max_norm=v)) == INVALID


def test_clip_refuses_overlapping_tensors():
    a, b = (4096, None, 100, 1), (8192, None, 100, 1)   # 400 bytes each
    for bad in ([a, a], [a, (4096 + 396, None, 4, 1)], [a, b, (4092, None, 2, 1)],
                [(4096, 8192, 100, 1), (8192, 16384, 100, 1)],   # one's output is another's input
                [(4096, 16384, 100, 1), (8192, 16384 + 200, 100, 1)],
                [(4096, 4096 + 200, 100, 1)]):                   # its own output, shifted
        assert _call("moe_grad_clip", _grad(bad)) == INVALID, bad
    many = [(4096 + 400 * i, None, 100, 1) for i in range(500)]
    assert _call("moe_grad_clip", _grad(many + [many[17]])) == INVALID


@no_device
def test_grad_accepts():
    for fn in ("moe_grad_sumsq", "moe_grad_clip"):
        many = [(4096 + 400 * i, None, 100, 1) for i in range(500)]
        for ok in ([], [(64, None, 4, 1)], [(None, None, 0, 0)], [(66, None, 4, 0)], many,
                   [(4096, 8192, 100, 1), (4096, 16384, 100, 1)]):
            assert _call(fn, _grad(ok)) == DEVICE, (fn, ok)
    assert _call("moe_grad_clip", _grad([(64, None, 4, 1)], max_norm=INF)) == DEVICE


def test_workspace_sizes():
    assert m.moe_router_loss_workspace_size(0, 4) > 0
    assert m.moe_router_loss_workspace_size(-1, 4) == 0 == m.moe_router_loss_workspace_size(4, 0)
    assert m.moe_router_loss_workspace_size(10 ** 6, 1024) >= m.moe_router_loss_workspace_size(10, 1024)
    assert m.moe_grad_workspace_size(0) > 0 and m.moe_grad_workspace_size(-1) == 0
    assert m.moe_grad_workspace_size(1000) > m.moe_grad_workspace_size(10)


def test_binding_refuses_other_tensors():
    """What the C side cannot see: types, sizes, strides, the device."""
    f32, bf = torch.zeros(4, 8), torch.zeros(16, 16, dtype=torch.bfloat16)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    both = dict(T=4, E=8, k=2, expert_idx=idx)
    import unittest.mock as mock
    with mock.patch.object(B, "_device", lambda: (B._setup(), 0)[1]):
        for logits in (f32.double(), torch.zeros(4, 7), torch.zeros(8, 4).t(), f32, "x"):   # the last tensor: not on a device
            with pytest.raises(ValueError):
                m.moe_router_bwd(**both, logits=logits, dlogits=f32)
        with pytest.raises(ValueError):
            m.moe_quantize_fp8(mode=m.QUANT_ROW, batch=1, rows=16, cols=16, x=bf.float(), q=bf, s=f32)
        with pytest.raises(ValueError):
            m.moe_grad_sumsq(tensors=[torch.zeros(3, dtype=torch.float16)], sumsq=f32, workspace=f32)
        with pytest.raises(ValueError):
            m.moe_grad_clip(tensors=[f32], out=[], sumsq=f32, max_norm=1.0)
        with pytest.raises(ValueError):
            m.moe_grad_clip(tensors=[f32], out=[f32.double()], sumsq=f32, max_norm=1.0)


def test_binding_refuses_other_arguments():
    """Numbers that do not fit, lists that are none, sizes whose product passes
    64 bits: exceptions, never a wrapped number."""
    import unittest.mock as mock
    f32 = torch.zeros(4, 8)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    bf = torch.zeros(16, 16, dtype=torch.bfloat16)
    with mock.patch.object(B, "_device", lambda: (B._setup(), -1)[1]):   # -1: the CPU tensors' device
        with pytest.raises(OverflowError):
            m.moe_router_bwd(T=2 ** 32 + 4, E=8, k=2, expert_idx=idx, logits=f32, dlogits=f32)
        with pytest.raises(OverflowError):
            m.moe_router_bwd(T=2 ** 70, E=8, k=2, expert_idx=idx, logits=f32, dlogits=f32)
        for T in ("4", 4.5, None):
            with pytest.raises(TypeError):
                m.moe_router_bwd(T=T, E=8, k=2, expert_idx=idx, logits=f32, dlogits=f32)
        big = 2 ** 31 - 1
        with pytest.raises(ValueError, match="x must be a contiguous tensor of type torch.bfloat16"):
            m.moe_quantize_fp8(mode=m.QUANT_ROW, batch=big, rows=big, cols=big, x=bf, q=f32, s=f32)
        for tensors in (None, 3, [None], ["x"], [f32, 1]):
            with pytest.raises(ValueError):
                m.moe_grad_sumsq(tensors=tensors, sumsq=torch.zeros(1, dtype=torch.float64),
                                 workspace=torch.zeros(64, dtype=torch.uint8))
        with pytest.raises(ValueError):   # a layout that is no strided one
            m.moe_grad_clip(tensors=[f32.to_sparse()], sumsq=torch.zeros(1, dtype=torch.float64), max_norm=1.0)
        with pytest.raises(m.MoeError):   # what the library itself refuses
            m.moe_router_bwd(T=-1, E=8, k=2, expert_idx=idx, logits=f32, dlogits=f32, stream=0)
        with pytest.raises(AttributeError):
            m.moe_router_bwd(T=4, E=8, k=2, expert_idx=idx, logits=f32, dlogits=f32, stream="x")


@no_device
def test_sizes_past_a_launch():
    """Grids that a launch cannot hold are refused; the largest that fit are not."""
    for mode, rows, cols, want in ((m.QUANT_ROW, 2 ** 31 - 1, 16, UNSUPPORTED),
                                   (m.QUANT_ROW, 2 ** 28 - 16, 1024, DEVICE),
                                   (m.QUANT_BOTH, 2 ** 31 - 128, 16, DEVICE),
                                   (m.QUANT_BOTH, 2 ** 31 - 128, 144, UNSUPPORTED)):
        a = B.QuantFp8Args(mode, 1, rows, cols, 0, 4096, 8192, 64, 4096, 64, 0, None, None)
        assert _call("moe_quantize_fp8", a) == want, (mode, rows, cols)


def test_binding_refuses_a_stream_of_another_device():
    import types
    import unittest.mock as mock
    f32, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with mock.patch.object(B, "_device", lambda: (B._setup(), -1)[1]):
        with pytest.raises(ValueError, match="another device"):
            m.moe_router_bwd(T=4, E=8, k=2, expert_idx=idx, logits=f32, dlogits=f32,
                             stream=types.SimpleNamespace(cuda_stream=0, device_index=3))
        neg = torch.zeros(32, dtype=torch.complex64).conj().imag   # a pending negation
        assert neg.is_neg()
        with pytest.raises(ValueError):
            m.moe_grad_sumsq(tensors=[neg], sumsq=torch.zeros(1, dtype=torch.float64),
                             workspace=torch.zeros(64, dtype=torch.uint8))
