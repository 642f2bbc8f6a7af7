"""Global gradient norm and clipping (moe_grad_sumsq, moe_grad_clip) against
float64 through the C ABI.

Tolerances: the sum of squares adds n exact fp64 squares, each addition off by
half an fp64 step at most (n 2^-53 relative, all terms positive); the factor
is rounded once to fp32, the product once (2 * 2^-24 relative), and a bf16
result once more (2^-8)."""

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import step as st

pytestmark = pytest.mark.gpu

DEV = "cuda"


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _sumsq(grads, ws=None):
    s = torch.full((1,), float("nan"), dtype=torch.float64, device=DEV)
    if ws is None:
        ws = torch.full((mg.moe_grad_workspace_size(len(grads)),), 0xFF, dtype=torch.uint8, device=DEV)
    mg.moe_grad_sumsq(tensors=grads, sumsq=s, workspace=ws)
    return s


def _check_clip(grads, got, f):
    for g, o in zip(grads, got):
        ref = g.double() * f
        tol = ref.abs() * ((2.0 ** -8 if g.dtype == torch.bfloat16 else 0) + 2.0 ** -22)
        # below the normal range a step is absolute: half of 2^-133 or 2^-149
        tol = tol + (2.0 ** -134 if g.dtype == torch.bfloat16 else 2.0 ** -150) * 1.01
        bad = int((~((o.double() - ref).abs() <= tol)).sum())
        assert bad == 0, f"{bad} of {g.numel()} values off"


def _make(sizes, seed=0, scale=1e-2, types=(torch.bfloat16, torch.float32)):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(n, generator=g, device=DEV) * scale).to(types[i % len(types)])
            for i, n in enumerate(sizes)]


LISTS = {
    "one_value": [1],
    "small_odd": [1, 7, 8, 9, 15, 17, 63, 127, 1000, 3],
    "chunk_edges": [16383, 16384, 16385, 16391, 16392, 32768, 32775, 49152],
    "with_empty": [0, 5, 0, 0, 4097, 0],
    "all_empty": [0, 0],
    "none": [],
    "more_than_one_launch": [3 + i % 50 for i in range(300)],
    "large": [5_000_003, 2_000_000],
}


@pytest.mark.parametrize("types", [(torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clip(name, types):
    grads = _make(LISTS[name], types=types)
    s = _sumsq(grads)
    ref = sum(float((g.double() ** 2).sum()) for g in grads)
    n = sum(LISTS[name])
    assert abs(s.item() - ref) <= 4 * max(n, 1) * 2.0 ** -53 * ref
    norm = torch.empty(1, device=DEV)
    for max_norm in (0.0, 0.37 * ref ** 0.5, 2 * ref ** 0.5 + 1, float("inf")):
        f = st.clip_factor(ref ** 0.5, max_norm)
        out = [torch.full_like(g, float("nan")) for g in grads]
        mg.moe_grad_clip(tensors=grads, out=out, sumsq=s, max_norm=max_norm, norm=norm)
        assert abs(norm.item() - ref ** 0.5) <= 2.0 ** -24 * 1.01 * ref ** 0.5
        _check_clip(grads, out, f)
        inplace = [g.clone() for g in grads]
        mg.moe_grad_clip(tensors=inplace, sumsq=s, max_norm=max_norm)
        for a, b in zip(out, inplace):
            assert torch.equal(a, b)


@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (1, 0), (0, 3), (5, 2), (7, 7)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_unaligned_slices_leave_their_neighbours(a, b, dt):
    n = 40001
    src = _make([n + 16], types=(dt,))[0]
    dst = torch.full((n + 16,), 5.0, dtype=dt, device=DEV)
    g, o = src[a:a + n], dst[b:b + n]
    s = _sumsq([g])
    ref = float((g.double() ** 2).sum())
    assert abs(s.item() - ref) <= 4 * n * 2.0 ** -53 * ref
    keep = src.clone()
    mg.moe_grad_clip(tensors=[g], out=[o], sumsq=s, max_norm=0.5 * ref ** 0.5)
    assert torch.equal(src, keep)
    _check_clip([g], [o], st.clip_factor(ref ** 0.5, 0.5 * ref ** 0.5))
    assert (dst[:b] == 5).all() and (dst[b + n:] == 5).all()
    mg.moe_grad_clip(tensors=[g], sumsq=s, max_norm=0.5 * ref ** 0.5)
    assert torch.equal(g, o)
    assert torch.equal(src[:a], keep[:a]) and torch.equal(src[a + n:], keep[a + n:])


def test_squares_past_the_fp32_range():
    """Gradients whose squares leave fp32 at both ends."""
    for v in (1e30, 1e-30):
        g = torch.full((1000,), v, dtype=torch.float32, device=DEV)
        s = _sumsq([g])
        ref = 1000 * float(g[0].double()) ** 2
        assert abs(s.item() - ref) <= 1e-12 * ref
        norm = torch.empty(1, device=DEV)
        out = torch.empty_like(g)
        mg.moe_grad_clip(tensors=[g], out=[out], sumsq=s, max_norm=1e-31, norm=norm)
        _check_clip([g], [out], st.clip_factor(ref ** 0.5, float(np.float32(1e-31))))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    grads = _make([100, 3000])
    grads[1][17] = bad
    s = _sumsq(grads)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    norm = torch.empty(1, device=DEV)
    out = [torch.empty_like(g) for g in grads]
    mg.moe_grad_clip(tensors=grads, out=out, sumsq=s, max_norm=1e-3, norm=norm, err_flag=err)
    assert err.item() == mg.DEVERR_NONFINITE
    assert not np.isfinite(norm.item())
    for g, o in zip(grads, out):
        assert torch.equal(g.view(torch.int16 if g.dtype == torch.bfloat16 else torch.int32),
                           o.view(torch.int16 if g.dtype == torch.bfloat16 else torch.int32)) or bad != bad
    same = [g.clone() for g in grads]
    mg.moe_grad_clip(tensors=same, sumsq=s, max_norm=1e-3)
    torch.cuda.synchronize()
    for g, o in zip(grads, same):   # in place: not even a NaN's bits change
        bits = torch.int16 if g.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(g.view(bits), o.view(bits))


def test_the_same_tensor_twice():
    g = _make([1000])[0]
    s = _sumsq([g, g])   # counted twice
    ref = 2 * float((g.double() ** 2).sum())
    assert abs(s.item() - ref) <= 1e-10 * ref
    for tensors, out in (([g, g], None), ([g, g[10:20]], None), ([g[:500], g[600:]], [g[500:], g[:400]])):
        with pytest.raises((mg.MoeError, ValueError)):
            mg.moe_grad_clip(tensors=tensors, out=out, sumsq=s, max_norm=1.0)
    # the same input into two outputs is fine
    o = [torch.empty_like(g), torch.empty_like(g)]
    mg.moe_grad_clip(tensors=[g, g], out=o, sumsq=s, max_norm=1e9)
    assert torch.equal(o[0], g) and torch.equal(o[1], g)


def test_graph_replays_same_bits_and_offsets_past_32_bits():
    big = torch.empty((1 << 31) + 1000, dtype=torch.bfloat16, device=DEV)
    big.fill_(2.0 ** -10)
    big[-1] = 3.0
    s = _sumsq([big])
    ref = ((1 << 31) + 999) * 2.0 ** -20 + 9.0
    assert abs(s.item() - ref) <= 1e-9 * ref
    mg.moe_grad_clip(tensors=[big], sumsq=s, max_norm=0.5 * ref ** 0.5)
    f = st.clip_factor(ref ** 0.5, 0.5 * ref ** 0.5)
    for i in (0, 1 << 30, (1 << 31) - 1, (1 << 31) + 998):
        assert abs(big[i].item() - 2.0 ** -10 * f) <= (2.0 ** -8 + 2.0 ** -22) * 2.0 ** -10 * f
    assert abs(big[-1].item() - 3.0 * f) <= (2.0 ** -8 + 2.0 ** -22) * 3 * f
    del big
    grads = _make([10_000, 333, 70_000])
    work = [torch.empty_like(g) for g in grads]
    s, norm = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(1, device=DEV)
    ws = torch.empty(mg.moe_grad_workspace_size(len(grads)), dtype=torch.uint8, device=DEV)

    def step():
        mg.moe_grad_sumsq(tensors=work, sumsq=s, workspace=ws)
        mg.moe_grad_clip(tensors=work, sumsq=s, max_norm=0.1, norm=norm)

    def eager():
        for w, g in zip(work, grads):
            w.copy_(g)
        step()
        torch.cuda.synchronize()
        return [w.clone() for w in work], s.item(), norm.item()

    ref = eager()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for _ in range(3):
        for w, x in zip(work, grads):
            w.copy_(x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(work, ref[0]))
        assert s.item() == ref[1] and norm.item() == ref[2]
        again = eager()
        assert all(torch.equal(a, b) for a, b in zip(again[0], ref[0])) and again[1:] == ref[1:]
