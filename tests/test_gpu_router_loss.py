"""The router's losses, counts and gradient (moe_router_loss, moe_router_bwd)
against the float64 oracle through the C ABI.

Tolerances (u = 2^-24, half an fp32 step).  A probability is expf(x - m) / z:
the difference is rounded (|x - m| u relative, below 64 u for the logits used
here, whose spread stays under 64), expf and the division are within 4 u, and
z is a sum of at most 16 terms a lane and 6 exchanges of such numbers (22 u
more): p is within 100 u.  A gradient element is p times a sum of terms that
carry the same error and at most 30 additions, so it is within 400 u of the
sum of its terms' magnitudes, which the oracle returns; the mean and the
losses add fp32 sums over a workgroup's tokens (at most 256 additions for the
sizes here)."""

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import step as st

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _case(T, E, k, seed, masked=0.0):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, E)) + 1.4 * rng.standard_normal((1, E))).astype(np.float32)
    idx = np.argsort(-x, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = (rng.random(T) >= masked).astype(np.uint8) if masked else None
    dprobs = rng.standard_normal((T, k)).astype(np.float32)
    return x, idx, mask, dprobs


def _up(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _loss(x, idx, mask, balance, zc, offset=0):
    T, E = x.shape
    k = idx.shape[1]
    lg = torch.empty(T * E + 4, device=DEV)
    lg = lg[offset:offset + T * E].view(T, E)   # offset 1: rows that no 16-byte load may start
    lg.copy_(_up(x))
    out = dict(counts=torch.full((E,), -1, dtype=torch.int32, device=DEV),
               n_tokens=torch.full((1,), -1, dtype=torch.int32, device=DEV),
               prob_mean=torch.full((E,), -1.0, device=DEV), loss=torch.full((2,), -1.0, device=DEV))
    ws = torch.full((mg.moe_router_loss_workspace_size(T, E),), 0xFF, dtype=torch.uint8, device=DEV)
    mg.moe_router_loss(T=T, E=E, k=k, logits=lg, expert_idx=_up(idx), token_mask=_up(mask),
                       balance_coef=balance, z_coef=zc, workspace=ws, **out)
    torch.cuda.synchronize()
    return lg, out


def _bwd(lg, idx, mask, balance, zc, out, dprobs=None, dloss=None):
    T, E = lg.shape
    d = torch.full((T, E), float("nan"), device=DEV)
    mg.moe_router_bwd(T=T, E=E, k=idx.shape[1], logits=lg, expert_idx=_up(idx), token_mask=_up(mask),
                      balance_coef=balance, z_coef=zc, counts=out and out["counts"],
                      n_tokens=out and out["n_tokens"], dprobs=_up(dprobs), dloss=_up(dloss), dlogits=d)
    torch.cuda.synchronize()
    return d.double().cpu().numpy()


def _check(x, idx, mask, dprobs, balance=0.3, zc=0.2, dloss=None, offset=0):
    lg, out = _loss(x, idx, mask, balance, zc, offset)
    counts, n, mean, loss = st.router_loss(x, idx, mask, balance, zc)
    np.testing.assert_array_equal(out["counts"].cpu().numpy(), counts)
    assert out["n_tokens"].item() == n
    np.testing.assert_allclose(out["prob_mean"].double().cpu().numpy(), mean, rtol=400 * U, atol=0)
    np.testing.assert_allclose(out["loss"].double().cpu().numpy(), loss, rtol=800 * U, atol=0)
    d = _bwd(lg, idx, mask, balance, zc, out, dprobs, dloss)
    ref, scale = st.router_bwd(x, idx, dprobs, dloss, counts, n, mask, balance, zc)
    bad = ~(np.abs(d - ref) <= 400 * U * scale + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:3], d[bad][:3], ref[bad][:3], scale[bad][:3])


CASES = [(1, 1, 1), (1, 2, 2), (3, 5, 1), (256, 4, 2), (777, 16, 8), (100, 17, 3), (511, 64, 6),
         (130, 65, 8), (64, 256, 8), (999, 250, 4), (40, 257, 2), (37, 1024, 8), (9, 1023, 1), (20000, 8, 2)]


@pytest.mark.parametrize("masked", [0.0, 0.4])
@pytest.mark.parametrize("T,E,k", CASES)
def test_losses_and_gradient(T, E, k, masked):
    x, idx, mask, dprobs = _case(T, E, k, T + E, masked)
    _check(x, idx, mask, dprobs, dloss=np.array([1.7, -0.6], np.float32))


@pytest.mark.parametrize("T,E,k", [(100, 64, 2), (33, 256, 8)])
def test_unaligned_logits(T, E, k):
    x, idx, mask, dprobs = _case(T, E, k, 5)
    _check(x, idx, mask, dprobs, offset=1)


def test_each_term_alone_and_defaults():
    x, idx, mask, dprobs = _case(300, 24, 3, 7, 0.2)
    _check(x, idx, mask, dprobs, balance=0.0, zc=0.0)
    _check(x, idx, mask, None, balance=0.5, zc=0.0)
    _check(x, idx, mask, None, balance=0.0, zc=0.5)
    # without coefficients counts are not needed, without dprobs all is zero
    lg = _up(x)
    assert not _bwd(lg, idx, mask, 0.0, 0.0, None).any()
    d = _bwd(lg, idx, mask, 0.0, 0.0, None, dprobs)
    ref, scale = st.router_bwd(x, idx, dprobs)
    assert (np.abs(d - ref) <= 400 * U * scale).all()


def test_everything_masked():
    x, idx, _, dprobs = _case(50, 12, 2, 8)
    mask = np.zeros(50, np.uint8)
    _, out = _loss(x, idx, mask, 0.3, 0.2)
    assert out["n_tokens"].item() == 0 and not out["counts"].any() and not out["prob_mean"].any()
    assert not out["loss"].any()
    _check(x, idx, mask, dprobs)


def test_no_tokens():
    out = _loss(np.zeros((0, 6), np.float32), np.zeros((0, 2), np.int32), None, 0.3, 0.2)[1]
    assert out["n_tokens"].item() == 0 and not out["counts"].any() and not out["loss"].any()


def test_dropped_and_repeated_picks():
    x, idx, mask, dprobs = _case(200, 20, 4, 9, 0.3)
    idx[::3, 1] = -1
    idx[1::3, 2] = 20
    idx[2::3, 3] = idx[2::3, 0]
    _check(x, idx, mask, dprobs)


def test_infinite_and_extreme_logits():
    x, idx, mask, dprobs = _case(64, 40, 2, 10)
    x[3] = -np.inf                      # no expert at all: left out, zero gradient
    x[4, 5:] = -np.inf                  # most experts ruled out
    x[5, :] = np.finfo(np.float32).min  # a mask of the type's lowest value everywhere
    x[6, 1:] = np.finfo(np.float32).min
    x[7] = 60 * (np.arange(40) % 2)
    idx[3] = [0, 1]
    idx[4] = [0, 1]
    balance, zc = 0.3, 0.0              # lse of row 5 squared would not be finite
    lg, out = _loss(x, idx, mask, balance, zc)
    counts, n, mean, loss = st.router_loss(x, idx, mask, balance, zc)
    assert n == 63 and out["n_tokens"].item() == 63
    np.testing.assert_array_equal(out["counts"].cpu().numpy(), counts)
    np.testing.assert_allclose(out["prob_mean"].double().cpu().numpy(), mean, rtol=400 * U)
    assert abs(out["loss"][0].item() - loss[0]) <= 800 * U * loss[0]
    d = _bwd(lg, idx, mask, balance, zc, out, dprobs)
    ref, scale = st.router_bwd(x, idx, dprobs, None, counts, n, mask, balance, zc)
    assert not d[3].any()
    assert (np.abs(d - ref) <= 400 * U * scale + 1e-37).all()


def test_nan_stays_in_its_row():
    x, idx, mask, dprobs = _case(40, 30, 2, 11)
    x[7, 3] = np.nan
    lg, out = _loss(x, idx, mask, 0.3, 0.2)
    assert np.isnan(out["loss"].cpu().numpy()).all() and np.isnan(out["prob_mean"].cpu().numpy()).all()
    d = _bwd(lg, idx, mask, 0.3, 0.0, out, dprobs)
    assert np.isnan(d[7]).all() and np.isfinite(np.delete(d, 7, 0)).all()


def test_gradient_by_differences_of_the_losses():
    """Central differences of the kernel's own losses (fp32, so a wide step)."""
    T, E, k = 16, 6, 2
    x, idx, _, _ = _case(T, E, k, 12)
    lg, out = _loss(x, idx, None, 1.0, 1.0)
    d = _bwd(lg, idx, None, 1.0, 1.0, out)
    h = 2.0 ** -5
    for t, e in ((0, 0), (3, 5), (15, 2)):
        xp, xm = x.copy(), x.copy()
        xp[t, e] += h
        xm[t, e] -= h
        lp = _loss(xp, idx, None, 1.0, 1.0)[1]["loss"].double().sum().item()
        lm = _loss(xm, idx, None, 1.0, 1.0)[1]["loss"].double().sum().item()
        # third derivative below 10 / T, losses of size 10 rounded to 2^-21
        assert abs((lp - lm) / (2 * h) - d[t, e]) <= 10 / T * h * h / 6 + 2.0 ** -20 / h


def test_graph_replays_and_same_bits():
    T, E, k = 3000, 128, 4
    x, idx, mask, dprobs = _case(T, E, k, 13, 0.1)
    lg, out = _loss(x, idx, mask, 0.3, 0.2)
    d = _bwd(lg, idx, mask, 0.3, 0.2, out, dprobs)
    bufs = dict(counts=torch.empty(E, dtype=torch.int32, device=DEV), n_tokens=torch.empty(1, dtype=torch.int32, device=DEV))
    pm, ls, dl = torch.empty(E, device=DEV), torch.empty(2, device=DEV), torch.empty(T, E, device=DEV)
    ws = torch.empty(mg.moe_router_loss_workspace_size(T, E), dtype=torch.uint8, device=DEV)
    lgd, ix, mk, dp = torch.empty_like(lg), _up(idx), _up(mask), _up(dprobs)
    both = dict(T=T, E=E, k=k, logits=lgd, expert_idx=ix, token_mask=mk, balance_coef=0.3, z_coef=0.2, **bufs)

    def step():
        mg.moe_router_loss(**both, prob_mean=pm, loss=ls, workspace=ws)
        mg.moe_router_bwd(**both, dprobs=dp, dlogits=dl)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for i in range(3):
        lgd.copy_(lg)
        dl.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs["counts"], out["counts"]) and torch.equal(pm, out["prob_mean"])
        assert torch.equal(ls, out["loss"])
        np.testing.assert_array_equal(dl.double().cpu().numpy(), d)
        lgd.zero_()
        step()
