"""Float64 oracle of the block-scaled FP8 products, the router's losses and
gradient, and the gradient norm with clipping.  Plain NumPy; shares no code
with the GPU path."""

from __future__ import annotations

import numpy as np

from . import numerics as nu

FP8_BLOCK = 128
SMALLEST = np.float32(2.0 ** -100)


# ------------------------------------------------------------ block FP8 ---
def block_scales(m: np.ndarray, pow2: bool = False):
    """(scale, factor of the codes), float32, of blocks with largest
    magnitudes m: m / 448 and 448 / m, each rounded once, or the smallest
    power of two not below m / 448 and its reciprocal."""
    m = np.maximum(m.astype(np.float32), SMALLEST)
    with np.errstate(over="ignore"):
        if not pow2:
            return m / np.float32(448), np.float32(448) / m
        f, e = np.frexp(m.astype(np.float64) / 448)     # m / 448 = f 2^e, f in [0.5, 1)
        e = np.where(f == 0.5, e - 1, e)
        s = np.where(np.isinf(m), np.float32(np.inf), np.ldexp(1.0, e).astype(np.float32))
        return s.astype(np.float32), (1.0 / s.astype(np.float64)).astype(np.float32)


def _amax(x, axes):
    """Largest magnitude; NaN does not count."""
    a = np.abs(x)
    return np.max(np.where(np.isnan(a), 0.0, a), axis=axes)


def quantize_rows(x: np.ndarray, pow2: bool = False):
    """x float64 [R][K] (bf16 values) -> codes uint8 [R][K], scales float32
    [ceil(K/128)][R]."""
    R, K = x.shape
    q = np.empty((R, K), dtype=np.uint8)
    s = np.empty((-(-K // FP8_BLOCK), R), dtype=np.float32)
    for b in range(s.shape[0]):
        sl = slice(b * FP8_BLOCK, min(K, (b + 1) * FP8_BLOCK))
        s[b], r = block_scales(_amax(x[:, sl], 1), pow2)
        with np.errstate(invalid="ignore"):
            q[:, sl] = nu.e4m3_encode((x[:, sl].astype(np.float32) * r[:, None]).astype(np.float64))
    return q, s


def quantize_tiles(x: np.ndarray, pow2: bool = False):
    """x float64 [R][K] -> codes [R][K], scales [ceil(R/128)][ceil(K/128)]."""
    R, K = x.shape
    q = np.empty((R, K), dtype=np.uint8)
    s = np.empty((-(-R // FP8_BLOCK), -(-K // FP8_BLOCK)), dtype=np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            t = (slice(i * FP8_BLOCK, (i + 1) * FP8_BLOCK), slice(j * FP8_BLOCK, (j + 1) * FP8_BLOCK))
            s[i, j], r = block_scales(_amax(x[t], (0, 1)), pow2)
            with np.errstate(invalid="ignore"):
                q[t] = nu.e4m3_encode((x[t].astype(np.float32) * r).astype(np.float64))
    return q, s


def dequantize_rows(q, s):
    v = nu.e4m3_decode(q)
    return v * np.repeat(s.astype(np.float64).T, FP8_BLOCK, axis=1)[:, :v.shape[1]]


def dequantize_tiles(q, s):
    v = nu.e4m3_decode(q)
    sp = np.repeat(np.repeat(s.astype(np.float64), FP8_BLOCK, axis=0), FP8_BLOCK, axis=1)
    return v * sp[:v.shape[0], :v.shape[1]]


def grouped_product(a, w, sizes, starts):
    """(C, sum of magnitudes) for dequantized a [M][K] and w [E][N][K]; rows
    outside the groups are NaN."""
    M, N = a.shape[0], w.shape[1]
    c, mag = np.full((M, N), np.nan), np.zeros((M, N))
    for e, (n, o) in enumerate(zip(sizes, starts)):
        c[o:o + n] = a[o:o + n] @ w[e].T
        mag[o:o + n] = np.abs(a[o:o + n]) @ np.abs(w[e]).T
    return c, mag


def grouped_weight_grad(a, b, sizes, starts):
    """(C [E][P][Q], sum of magnitudes) for dequantized a [P][M], b [Q][M]
    over each group's span of whole 128-row blocks."""
    c = np.zeros((len(sizes), a.shape[0], b.shape[0]))
    mag = np.zeros_like(c)
    for e, (n, o) in enumerate(zip(sizes, starts)):
        m = -(-n // FP8_BLOCK) * FP8_BLOCK
        c[e] = a[:, o:o + m] @ b[:, o:o + m].T
        mag[e] = np.abs(a[:, o:o + m]) @ np.abs(b[:, o:o + m]).T
    return c, mag


# ---------------------------------------------------------- router losses ---
def _softmax(x):
    """p, lse and whether a row has any finite logit."""
    with np.errstate(invalid="ignore", divide="ignore"):
        m = x.max(axis=1, keepdims=True)
        any_ = m[:, 0] != -np.inf
        ex = np.where(any_[:, None], np.exp(x - np.where(any_[:, None], m, 0.0)), 0.0)
        z = ex.sum(axis=1, keepdims=True)
        p = np.where(any_[:, None], ex / np.where(any_[:, None], z, 1.0), 0.0)
        lse = np.where(any_, m[:, 0] + np.log(np.where(any_, z[:, 0], 1.0)), 0.0)
    return p, lse, any_


def router_loss(logits, idx, mask=None, balance=0.0, zc=0.0):
    """counts, n, prob_mean, (balance loss, z loss) in float64."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    p, lse, any_ = _softmax(x)
    keep = any_ & (np.ones(T, bool) if mask is None else np.asarray(mask, dtype=bool))
    n, k = int(keep.sum()), idx.shape[1]
    ids = idx[keep].reshape(-1)
    counts = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E).astype(np.int64)
    if n == 0:
        return counts, 0, np.zeros(E), (0.0, 0.0)
    mean = p[keep].sum(axis=0) / n
    return (counts, n, mean, (balance * E * float((counts / (k * n) * mean).sum()),
                              zc * float((lse[keep] ** 2).sum()) / n))


def router_bwd(logits, idx, dprobs=None, dloss=None, counts=None, n=0, mask=None, balance=0.0,
               zc=0.0):
    """(dlogits, error scale): the scale is the sum of the magnitudes of the
    terms each element is made of."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    k = idx.shape[1]
    p, lse, any_ = _softmax(x)
    keep = any_ & (np.ones(T, bool) if mask is None else np.asarray(mask, dtype=bool))
    g = (1.0, 1.0) if dloss is None else tuple(float(v) for v in dloss)
    v = np.zeros((T, E))
    zt = np.zeros(T)
    if n > 0:
        if counts is not None:
            v += np.where(keep[:, None], g[0] * balance * E * counts / (k * n * n), 0.0)
        zt = np.where(keep, g[1] * 2 * zc * lse / n, 0.0)
    if dprobs is not None:
        for s in range(k):
            ok = (idx[:, s] >= 0) & (idx[:, s] < E)
            v[np.flatnonzero(ok), idx[ok, s]] += dprobs[ok, s]
    dot = (p * v).sum(axis=1, keepdims=True)
    d = p * (v - dot + zt[:, None])
    scale = p * (np.abs(v) + (p * np.abs(v)).sum(axis=1, keepdims=True) + np.abs(zt)[:, None])
    return d, scale


# ------------------------------------------------------- gradient clipping ---
def grad_norm(grads):
    return float(np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads)))


def clip_factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(norm) else 1.0
