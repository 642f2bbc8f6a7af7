"""Float64 oracle of the router's choice by scores and its gradient, of AdamW,
and of the 8-bit integer products.  Plain NumPy; shares no code with the GPU
path."""

from __future__ import annotations

import numpy as np

from . import numerics as nu

BLOCK = 128
SMALLEST = np.float32(2.0 ** -100)
INF = np.inf


# ------------------------------------------------------------- the choice ---
def scores(x: np.ndarray, sigmoid: bool) -> np.ndarray:
    """Scores of float64 logits [T][E]; -inf and NaN have none (0)."""
    ok = x > -INF
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return np.where(ok, 1 / (1 + np.exp(-np.where(ok, x, 0))), 0.0)
        m = np.max(np.where(ok, x, -INF), axis=1, keepdims=True)
        e = np.where(ok, np.where(x == m, 1.0, np.exp(x - np.where(np.isfinite(m), m, 0))), 0.0)
        e = np.where((m == INF) & (x != m), 0.0, e)
    z = e.sum(1, keepdims=True)
    return e / np.where(z > 0, z, 1)


def gate(x, k, sigmoid=False, bias=None, n_groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0, mask=None):
    """(expert_idx int64 [T][k] with -1, probs float64 [T][k]), one token and
    one pick after the other."""
    T, E = x.shape
    s = scores(x, sigmoid)
    judged = s if bias is None else s + bias.astype(np.float64)
    idx, w = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        choice = (x if bias is None else judged)[t].copy()
        choice[~((x[t] > -INF) & (judged[t] > -INF))] = -INF
        if n_groups > 1 and topk_groups < n_groups:
            value = []
            for g in range(n_groups):
                ids = range(g * E // n_groups, (g + 1) * E // n_groups)
                of = sorted((judged[t][e] if group_top == 2 else choice[e] for e in ids if choice[e] > -INF), reverse=True)
                value.append(sum(of[:group_top]) if of else -INF)
            stay = sorted(range(n_groups), key=lambda g: (-value[g], g))[:topk_groups]
            for g in set(range(n_groups)) - set(stay):
                choice[g * E // n_groups:(g + 1) * E // n_groups] = -INF
        picks = [e for e in sorted(range(E), key=lambda e: (-choice[e], e))[:k] if choice[e] > -INF]
        idx[t, :len(picks)] = picks
        w[t, :len(picks)] = weights(x[t][picks], s[t][picks], sigmoid, renorm)
    return idx, scale * w


def weights(x, s, sigmoid, renorm):
    """The picks' weights from their logits and scores."""
    if not renorm or not len(x):
        return s
    if sigmoid:   # in logarithms: all scores may be tiny
        log = np.where(x > 0, -np.log1p(np.exp(-np.abs(x))), np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x))))
    else:
        log = x
    e = np.where(log == log.max(), 1.0, np.exp(log - (log.max() if np.isfinite(log.max()) else 0)))
    e = np.where((log.max() == INF) & (log != INF), 0.0, e)
    return e / e.sum()


def gate_bwd(x, idx, dprobs, sigmoid=False, renorm=False, scale=1.0):
    """(dlogits float64 [T][E], the sums of the magnitudes that make it)."""
    T, E = x.shape
    s = scores(x, sigmoid)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        live = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E and x[t, idx[t, j]] > -INF]
        ids, g = idx[t, live], scale * dprobs[t, live]
        xs, sp = x[t, ids], s[t, ids]
        rest = scores(-xs[None], True)[0]   # 1 - sp of a sigmoid, also where sp rounds to 1
        if renorm:
            w = weights(xs, sp, sigmoid, True)
            part, parts = w * (g - (w * g).sum()), w * (np.abs(g) + (w * np.abs(g)).sum())
            if sigmoid:
                part, parts = part * rest, parts * rest
        elif sigmoid:
            part = g * sp * rest
            parts = np.abs(part)
        else:
            part, parts = g * sp, np.abs(g) * sp
            d[t] -= s[t] * part.sum()
            mag[t] += s[t] * parts.sum()
        np.add.at(d[t], ids, part)
        np.add.at(mag[t], ids, parts)
    return d, mag


def bias_update(counts, bias, rate):
    n = counts.astype(np.int64) * len(counts)
    return bias + np.float32(rate) * np.sign(counts.astype(np.int64).sum() - n).astype(np.float32)


# ------------------------------------------------------------------ AdamW ---
def mix32(x: int) -> int:
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random16(seed, step, tensor, n):
    key = mix32((mix32((seed + step * 0x9E3779B9) & 0xFFFFFFFF) + tensor) & 0xFFFFFFFF)
    h = [mix32((key + i) & 0xFFFFFFFF) for i in range((n + 1) // 2)]
    return np.array([h[i // 2] >> 16 if i & 1 else h[i // 2] & 0xFFFF for i in range(n)], dtype=np.float64)


def clip_factor(sumsq, max_norm):
    return 1.0 if sumsq is None else min(1.0, max_norm / (np.sqrt(sumsq) + 1e-6))


def adamw(w, g, m, v, lr, beta1, beta2, eps, wd, step, f=1.0):
    """float64 (w, m, v, |b1 m| + |a1 d|, the update's denominator)."""
    d = g * f
    m1, v1 = beta1 * m + (1 - beta1) * d, beta2 * v + (1 - beta2) * d * d
    den = np.sqrt(v1 / (1 - beta2 ** step)) + eps
    return (w - lr * wd * w - lr * m1 / (1 - beta1 ** step) / den, m1, v1, np.abs(beta1 * m) + np.abs((1 - beta1) * d), den)


def block_scale(x):
    """Scales (float64) of the blocks of a flat state."""
    n = -(-len(x) // BLOCK)
    p = np.zeros(n * BLOCK)
    p[:len(x)] = np.abs(x)
    return np.maximum(p.reshape(n, BLOCK).max(1), SMALLEST) / 448


def spread(s, n):
    return np.repeat(np.asarray(s, dtype=np.float64), BLOCK)[:n]


def e4m3_step(mag):
    return np.exp2(np.floor(np.log2(np.maximum(mag, 2.0 ** -6))) - 3)


# --------------------------------------------------------- 8-bit integers ---
def quantize_int8(x: np.ndarray):
    """x float64 [R][K] (bf16 values) -> codes int8, scales float32 [R]."""
    x32 = x.astype(np.float32)
    bad = ~np.isfinite(x32).all(1)
    m = np.maximum(np.abs(np.where(bad[:, None], 0, x32)).max(1), SMALLEST).astype(np.float32)
    r = np.float32(127) / m
    q = np.rint(np.where(bad[:, None], np.float32(0), x32) * r[:, None]).astype(np.int8)
    return q, np.where(bad, np.float32(np.nan), m / np.float32(127))


def product_int8(a, a_s, b, b_s, sizes, starts, n_rows):
    """float32 [n_rows][N] as the operator defines it (exact sums, rounded to
    fp32, scaled by the token's and then the weight row's scale); rows outside
    the groups are NaN."""
    c = np.full((n_rows, b.shape[1]), np.nan, dtype=np.float32)
    for e, (n, o) in enumerate(zip(sizes, starts)):
        # (sums below 2^53 are exact in float64)
        s = (a[o:o + n].astype(np.float64) @ b[e].astype(np.float64).T).astype(np.float32)
        c[o:o + n] = s * a_s[o:o + n, None] * b_s[e][None, :]
    return c


def round_bf16(x: np.ndarray) -> np.ndarray:
    return nu.round_bf16(x.astype(np.float64))
