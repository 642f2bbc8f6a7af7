"""Host-side checks of the router's choice, AdamW and 8-bit integer entry points
(no GPU needed): struct layout, refusals before a device is touched, workspace
sizes.  The C calls pass placeholder addresses, so the ones that would be valid
run only where no HIP device is present."""

import ctypes
import shutil
import subprocess

import pytest

import moe_grouped_mlp_amd as m
from moe_grouped_mlp_amd import binding as B

from .test_abi import DEVICE, HEADER, INVALID, UNSUPPORTED, _call, no_device
from .test_step_abi import INF, NAN, _make, _refuses

STRUCTS = {
    "moe_gate_args": B.GateArgs,
    "moe_gate_bwd_args": B.GateBwdArgs,
    "moe_bias_update_args": B.BiasUpdateArgs,
    "moe_adamw_tensor": B.AdamwTensor,
    "moe_adamw_args": B.AdamwArgs,
    "moe_quant_int8_args": B.QuantInt8Args,
    "moe_gemm_int8_args": B.GemmInt8Args,
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
    assert f"MOE_SCORE_SOFTMAX = {m.SCORE_SOFTMAX}, MOE_SCORE_SIGMOID = {m.SCORE_SIGMOID}" in text
    assert f"MOE_STATE_F32 = {m.STATE_F32}, MOE_STATE_FP8 = {m.STATE_FP8}" in text


gate = _make(B.GateArgs, dict(T=16, E=64, k=8, logits_type=1, n_groups=8, topk_groups=2, group_top=2, scale=1.0, logits=64, expert_idx=64, probs=64))
bwd = _make(B.GateBwdArgs, dict(T=16, E=64, k=8, scale=1.0, logits=64, expert_idx=64, dprobs=64, dlogits=64))
bias = _make(B.BiasUpdateArgs, dict(E=8, rate=1e-3, counts=64, bias=64))
quant = _make(B.QuantInt8Args, dict(rows=4, cols=48, x=64, q=64, s=64))
gemm = _make(B.GemmInt8Args, dict(E=4, N=48, K=144, M_cap=512, split_sizes=64, padded_offsets=64, a=64, a_s=64, b=64, b_s=64, c=64))


def test_gate_refusals():
    _refuses("moe_router_gate", gate, [
        dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=4, k=5, n_groups=1), dict(T=1 << 28, k=8), dict(score=2),
        dict(score=-1), dict(n_groups=-1), dict(n_groups=65, E=65), dict(n_groups=7), dict(topk_groups=0), dict(topk_groups=9),
        dict(group_top=0), dict(group_top=3), dict(E=16, topk_groups=3, k=7), dict(scale=NAN), dict(scale=INF), dict(logits_type=2),
        dict(ld=63), dict(ld=-64), dict(logits=None), dict(expert_idx=None), dict(probs=None), dict(logits=66)])


@no_device
def test_gate_accepts():
    _refuses("moe_router_gate", gate, [
        dict(), dict(n_groups=0), dict(n_groups=1, topk_groups=0, group_top=0), dict(n_groups=64, topk_groups=64), dict(ld=70),
        dict(logits_type=0, logits=66), dict(bias=64, token_mask=64, counts=64), dict(T=0, logits=None, expert_idx=None, probs=None),
        dict(E=1024, n_groups=64, topk_groups=1)], DEVICE)


def test_gate_bwd_refusals():
    _refuses("moe_router_gate_bwd", bwd, [
        dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=4, k=5), dict(T=1 << 28, k=8), dict(score=2), dict(scale=NAN),
        dict(logits_type=-1), dict(ld=63), dict(ld_d=63), dict(logits=None), dict(expert_idx=None), dict(dprobs=None), dict(dlogits=None),
        dict(dlogits=65), dict(logits_type=1, dlogits=66)])


@no_device
def test_gate_bwd_accepts():
    _refuses("moe_router_gate_bwd", bwd, [
        dict(), dict(accumulate=1), dict(ld=64, ld_d=100), dict(T=0, logits=None, expert_idx=None, dprobs=None, dlogits=None)], DEVICE)


def test_bias_update_refusals():
    _refuses("moe_router_bias_update", bias, [dict(E=0), dict(E=1025), dict(rate=NAN), dict(rate=INF), dict(counts=None), dict(bias=None)])


def _adamw(tensors, /, **kw):
    arr = (B.AdamwTensor * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        for k, v in t.items():
            setattr(arr[i], k, v)
    a = B.AdamwArgs(arr, len(tensors), 0, 1e-3, 0.9, 0.999, 1e-8, 1, 1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _tensor(at=1 << 20, **kw):
    """100 elements, buffers 4096 bytes apart."""
    t = dict(param=at, grad=at + 4096, m=at + 8192, v=at + 12288, m_scale=at + 16384, v_scale=at + 20480, numel=100, param_type=1, grad_type=1)
    return {**t, **kw}


@pytest.mark.parametrize("state", [0, 1])
def test_adamw_refusals(state):
    at = 1 << 20
    for bad in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(numel=-1), dict(numel=1 << 47), dict(param_type=2),
                dict(grad_type=-1), dict(weight_decay=NAN), dict(weight_decay=INF), dict(master=at + 24576), dict(param=at + 2),
                dict(grad=at + 4097), dict(param_type=0, master=at + 24577),
                dict(m=at), dict(v=at + 8192 + 96), dict(grad=at + 396), dict(param_type=0, master=at + 100)):   # overlaps
        assert _call("moe_adamw", _adamw([_tensor(1 << 24), _tensor(**bad)], state_type=state)) == INVALID, bad
    for bad in (dict(m_scale=None), dict(v_scale=None), dict(m_scale=at + 2), dict(v_scale=at + 16384)) if state else (dict(m=at + 8194), dict(v=at + 12290)):
        assert _call("moe_adamw", _adamw([_tensor(**bad)], state_type=state)) == INVALID, bad
    for bad in (dict(n_tensors=-1), dict(tensors=None), dict(state_type=2), dict(lr=NAN), dict(lr=INF), dict(beta1=-0.1), dict(beta1=1.0),
                dict(beta2=1.0), dict(beta2=NAN), dict(eps=-1e-8), dict(eps=INF), dict(eps=NAN), dict(step=0), dict(step=-1),
                dict(sumsq=64, max_norm=-1.0), dict(sumsq=64, max_norm=NAN), dict(sumsq=68), dict(step_dev=66), dict(lr_dev=65)):
        assert _call("moe_adamw", _adamw([_tensor()], **{**dict(state_type=state), **bad})) == INVALID, bad
    assert _call("moe_adamw", _adamw([_tensor(), _tensor()], state_type=state)) == INVALID   # one tensor twice
    many = [_tensor((1 << 24) + i * 32768) for i in range(300)]
    assert _call("moe_adamw", _adamw([*many, _tensor((1 << 24) + 7 * 32768)], state_type=state)) == INVALID


@no_device
@pytest.mark.parametrize("state", [0, 1])
def test_adamw_accepts(state):
    many = [_tensor((1 << 24) + i * 32768) for i in range(300)]
    shared = [_tensor(1 << 24), _tensor(1 << 25, grad=(1 << 24) + 4096)]   # gradients may overlap
    for ok in ([], [_tensor()], [dict(numel=0, param_type=1)], many, shared, [_tensor(param_type=0, master=(1 << 20) + 24576)]):
        assert _call("moe_adamw", _adamw(ok, state_type=state)) == DEVICE
    assert _call("moe_adamw", _adamw([_tensor()], state_type=state, step=0, step_dev=64, lr_dev=64, sumsq=64, max_norm=INF)) == DEVICE


def test_quantize_refusals():
    _refuses("moe_quantize_int8", quant, [
        dict(rows=-1), dict(cols=0), dict(cols=8), dict(cols=40), dict(x=None), dict(q=None), dict(s=None), dict(x=72), dict(q=72),
        dict(x_stride=40), dict(x_stride=52), dict(x_stride=-48)])
    _refuses("moe_quantize_int8", quant, [dict(rows=1 << 24)], UNSUPPORTED)


@no_device
def test_quantize_accepts():
    _refuses("moe_quantize_int8", quant, [dict(), dict(x_stride=56), dict(rows=0, x=None, q=None, s=None), dict(row_end=64)], DEVICE)


def test_product_refusals():
    _refuses("moe_grouped_gemm_int8", gemm, [
        dict(E=0), dict(E=1025), dict(N=0), dict(N=40), dict(K=0), dict(K=100), dict(K=131072), dict(M_cap=0), dict(M_cap=1 << 31),
        dict(split_sizes=None), dict(padded_offsets=None), dict(a=None), dict(a_s=None), dict(b=None), dict(b_s=None), dict(c=None),
        dict(a=72), dict(b=72), dict(c=72), dict(workspace=72), dict(c_type=2), dict(c_type=-1), dict(max_rows=-1), dict(cu_margin=-1),
        dict(b_stride=48), dict(b_stride=48 * 144 + 8), dict(b_s_stride=47), dict(ldc=40), dict(ldc=52)])
    _refuses("moe_grouped_gemm_int8", gemm, [dict(M_cap=(1 << 31) - 1, N=1 << 30)], UNSUPPORTED)


@no_device
def test_product_accepts():
    _refuses("moe_grouped_gemm_int8", gemm, [
        dict(), dict(c_type=1), dict(max_rows=1), dict(ldc=56), dict(b_stride=48 * 144 + 16, b_s_stride=50), dict(M_cap=1), dict(K=131056)], DEVICE)


def test_workspace_sizes():
    assert m.moe_grouped_gemm_int8_workspace_size(2, 256, 8192, 512) > 0
    assert m.moe_grouped_gemm_int8_workspace_size(2, 256, 8192, 512, max_rows=16) == 0
    assert m.moe_grouped_gemm_int8_workspace_size(0, 256, 8192, 512) == 0


def test_more_tokens_than_a_launch_has_threads_for():
    for name, make in (("moe_router_gate", gate), ("moe_router_gate_bwd", bwd)):
        _refuses(name, make, [dict(T=1 << 26), dict(T=(1 << 27) - 1)], UNSUPPORTED)
