"""What the operators of a block-scaled 8-bit expert layer's training step and of its serving are measured on.

Five kinds of case, one operator each:

* ``quantize``: bf16 to E4M3 codes with an fp32 scale for each block of 128.
* ``gemm``: the grouped product of such activations and weights, for prompts, for training (forward and, on the
  transposed weights, the input's gradient) and for single tokens.
* ``wgrad``: the weights' gradient, the grouped product along the routed rows.
* ``balance``: the router's balance and z losses, the per-expert counts, and the gradient with respect to the logits.
* ``clip``: the global norm of a list of gradients, and the gradients scaled to a largest norm.

``own`` chooses between the plain form (elementary torch operations) and the library's kernels.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 128          # values that share a scale, and the alignment of a group's first row
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -100   # a block whose largest magnitude is below this is scaled as if it were this
F8 = torch.float8_e4m3fn
EPS = 1e-6           # added to the norm before the division of the clipping factor


def _up(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # the rows of one decoding step: 16 tokens' hidden vectors, where the call's latency counts
        dict(name="quantize rows decode", kind="quantize", mode="row", batch=1, rows=16, cols=4096, pow2=False),
        # the activations between the two products of a training step, row copies for the forward and transposed
        # ones for the weights' gradient, made together
        dict(name="quantize both activations", kind="quantize", mode="both", batch=1, rows=17408, cols=14336, pow2=False),
        # every expert's weights after an optimizer step; 2880 = 22.5 blocks, power-of-two scales
        dict(name="quantize tiles weights", kind="quantize", mode="tile", batch=128, rows=2880, cols=2880, pow2=True),
        # one decoding step of 8 tokens, two experts each: two rows for each of the 8 experts, the weights' bytes count
        dict(name="gemm decode", kind="gemm", E=8, k=2, T=8, N=28672, K=4096, skew="even", empty=0, out="bf16"),
        # the second product of a training step of a layer of 8 wide experts
        dict(name="gemm wide experts", kind="gemm", E=8, k=2, T=8192, N=4096, K=14336, skew="even", empty=0, out="bf16"),
        # the first product of a layer of many experts, unevenly loaded, 39 of them with no rows; K = 22.5 blocks
        dict(name="gemm many experts", kind="gemm", E=128, k=4, T=16384, N=5760, K=2880, skew="biased", empty=39, out="bf16"),
        # the weights' gradient of a small layer
        dict(name="wgrad small", kind="wgrad", E=4, k=2, T=256, P=512, Q=128, skew="even", empty=0, out="bf16"),
        # the weights' gradient of one device's share of a layer, very unequal groups, four of them empty, 32-bit sums
        dict(name="wgrad skewed share", kind="wgrad", E=32, k=1, T=16384, P=7168, Q=2048, skew="zipf", empty=4, out="f32"),
        # the router of a small layer: latency
        dict(name="balance small", kind="balance", T=256, E=4, k=2, masked=0.0, z=True),
        # the router of a layer of 256 experts over a padded batch
        dict(name="balance 256 experts", kind="balance", T=16384, E=256, k=8, masked=0.1, z=True),
        # sixty small gradients of odd sizes (norms, biases, routers), both types
        dict(name="clip many small", kind="clip", tensors=60, largest=200_001, dtype="mixed", clipped=True),
        # the two stacked weight gradients of a layer of 8 wide experts
        dict(name="clip expert weights", kind="clip", tensors=2, largest=8 * 28672 * 4096, dtype="bf16", clipped=True),
    ]


def _between(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    kind = rng.choice(("quantize", "gemm", "gemm", "wgrad", "balance", "clip"))
    if kind == "quantize":
        mode = rng.choice(("row", "both", "tile"))
        batch = _between(rng, 1, 64) if mode == "tile" else 1
        cols = _between(rng, 16, 16384, 16)
        rows = _between(rng, 1 if mode == "row" else 16, min(32768, max(64, (1 << 28) // (batch * cols))), 1 if mode == "row" else 16)
        return dict(kind=kind, mode=mode, batch=batch, rows=rows, cols=cols, pow2=rng.random() < 0.3)
    if kind in ("gemm", "wgrad"):
        E = _between(rng, 1, 96)
        k = rng.choice([j for j in (1, 2, 4, 8) if j <= E])
        empty = rng.choice((0, 0, E // 4)) if E - E // 4 >= k else 0
        T = _between(rng, 1, 8192)
        X = _between(rng, 64, 8192, 16)
        Y = _between(rng, 64, max(64, min(8192, (1 << 29) // (E * X))), 16)
        T = max(1, min(T, int(6e11 / (k * X * Y))))
        case = dict(kind=kind, E=E, k=k, T=T, skew=rng.choice(("even", "biased", "zipf")), empty=empty, out=rng.choice(("bf16", "f32")))
        return {**case, "N": X, "K": Y} if kind == "gemm" else {**case, "P": X, "Q": Y}
    if kind == "balance":
        E = _between(rng, 2, 1024)
        return dict(kind=kind, T=_between(rng, 1, max(1, min(65536, (1 << 22) // E))), E=E, k=rng.randint(1, min(8, E)),
                    masked=rng.choice((0.0, 0.1, 0.5)), z=rng.random() < 0.7)
    return dict(kind=kind, tensors=_between(rng, 1, 60), largest=_between(rng, 100, 20_000_000), dtype=rng.choice(("bf16", "f32", "mixed")),
                clipped=rng.random() < 0.8)


def _sizes(case):
    """Rows of each expert, largest first: the same for every seed (which expert has which goes by the seed)."""
    E, live, M = case["E"], case["E"] - case["empty"], case["T"] * case["k"]
    at = (np.arange(live) + 0.5) / live
    if case["skew"] == "zipf":
        w = 1.0 / np.arange(1, live + 1) ** 1.2
    elif case["skew"] == "biased":   # loads of a router whose experts' logits have normal offsets
        w = np.exp(1.5 * math.sqrt(2) * torch.erfinv(torch.from_numpy(1 - 2 * at)).numpy())
    else:
        w = np.ones(live)
    n = np.minimum(np.floor(M * w / w.sum()).astype(np.int64), case["T"])
    while n.sum() < M:               # what rounding left (and what a token's one row for an expert cut off)
        free = np.flatnonzero(n < case["T"])[: M - int(n.sum())]
        n[free] += 1
    return [int(v) for v in n] + [0] * (E - live)


def _clip_sizes(case):
    r = random.Random(case["tensors"] * 1_000_003 + case["largest"])
    sizes = [case["largest"]]
    while len(sizes) < case["tensors"]:
        sizes.append(case["largest"] // 2 if case["tensors"] == 2 else _between(r, 1, case["largest"]))
    kinds = {"bf16": (torch.bfloat16,), "f32": (torch.float32,), "mixed": (torch.bfloat16, torch.float32)}[case["dtype"]]
    return [(n, kinds[i % len(kinds)]) for i, n in enumerate(sizes)]


def work(case):
    c = case
    if c["kind"] == "quantize":
        n = c["batch"] * c["rows"] * c["cols"]
        copies = 1 if c["mode"] == "row" else 2
        per_scale = BLOCK * BLOCK if c["mode"] == "tile" else BLOCK
        return dict(bytes=2 * n + copies * (n + 4 * n / per_scale), flops=2 * n)
    if c["kind"] == "gemm":
        sizes = _sizes(c)
        M, live = sum(sizes), sum(n > 0 for n in sizes)
        return dict(bytes=M * c["K"] * (1 + 4 / BLOCK) + live * c["N"] * c["K"] + M * c["N"] * (4 if c["out"] == "f32" else 2),
                    flops=2 * M * c["N"] * c["K"])
    if c["kind"] == "wgrad":
        M = sum(_sizes(c))
        return dict(bytes=M * (c["P"] + c["Q"]) * (1 + 4 / BLOCK) + c["E"] * c["P"] * c["Q"] * (4 if c["out"] == "f32" else 2),
                    flops=2 * M * c["P"] * c["Q"])
    if c["kind"] == "balance":
        n = c["T"] * c["E"]
        return dict(bytes=2 * 4 * n + 8 * c["T"] * c["k"], flops=20 * n)
    total = sum(n * (2 if t == torch.bfloat16 else 4) for n, t in _clip_sizes(c))
    return dict(bytes=2 * total, flops=3 * sum(n for n, _ in _clip_sizes(c)))


# ------------------------------------------------------------- preparation --
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _scale_of(m, pow2):
    """(scale, its reciprocal) of blocks with the largest magnitudes m (fp32): m / 448, or the next power of two, in 64 bits, rounded once."""
    m = m.clamp(min=SMALLEST).double()
    s = m / E4M3_MAX
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
        return s.float(), (1 / s).float()
    return s.float(), (E4M3_MAX / m).float()


def _quantize_rows(x, pow2=False):
    """x [R][K] -> codes [R][K], scales [ceil(K / 128)][R]."""
    R, K = x.shape
    nb = -(-K // BLOCK)
    v = torch.zeros(R, nb * BLOCK, dtype=torch.float32, device=x.device)
    v[:, :K] = x.float()
    v = v.view(R, nb, BLOCK)
    s, r = _scale_of(v.abs().amax(2), pow2)
    q = (v * r[:, :, None]).to(F8).view(R, nb * BLOCK)[:, :K].contiguous()
    return q, s.t().contiguous()


def _quantize_tiles(x, pow2=False):
    """x [R][K] -> codes [R][K], scales [ceil(R / 128)][ceil(K / 128)]."""
    R, K = x.shape
    nr, nb = -(-R // BLOCK), -(-K // BLOCK)
    v = torch.zeros(nr * BLOCK, nb * BLOCK, dtype=torch.float32, device=x.device)
    v[:R, :K] = x.float()
    v = v.view(nr, BLOCK, nb, BLOCK)
    s, r = _scale_of(v.abs().amax((1, 3)), pow2)
    q = (v * r[:, None, :, None]).to(F8).view(nr * BLOCK, nb * BLOCK)[:R, :K].contiguous()
    return q, s


def _groups(case, seed):
    sizes = _sizes(case)
    random.Random(seed).shuffle(sizes)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _up(n, BLOCK))
    return sizes, starts, _up(case["T"] * case["k"] + case["E"] * (BLOCK - 1), BLOCK)


def _rows(g, case, sizes, starts, M_cap, width):
    """Routed rows with the rows between groups zero, as the permutation leaves them; magnitudes differ by row and by column."""
    x = _randn(g, M_cap, width) * torch.exp(0.5 * _randn(g, M_cap, 1)) * torch.exp(0.5 * _randn(g, 1, width))
    keep = torch.zeros(M_cap, 1, dtype=torch.float32, device="cuda")
    for n, o in zip(sizes, starts):
        keep[o:o + n] = 1
    return (x * keep).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["kind"] == "quantize":
        b, R, K = c["batch"], c["rows"], c["cols"]
        x = torch.empty(b, R, K, dtype=torch.bfloat16, device="cuda")
        for i in range(b):
            x[i] = (_randn(g, R, K) * torch.exp(_randn(g, R, 1))).to(torch.bfloat16)
        nb, nr = -(-K // BLOCK), -(-R // BLOCK)
        u8, f32 = dict(dtype=torch.uint8, device="cuda"), dict(dtype=torch.float32, device="cuda")
        c.update(x=x, q=torch.empty(b, R, K, **u8))
        c["s"] = torch.empty(b, nr, nb, **f32) if c["mode"] == "tile" else torch.empty(b, nb, R, **f32)
        if c["mode"] != "row":
            c["qT"] = torch.empty(b, K, R, **u8)
            c["sT"] = torch.empty(b, nb, nr, **f32) if c["mode"] == "tile" else torch.empty(b, nr, K, **f32)
        return c
    if c["kind"] in ("gemm", "wgrad"):
        sizes, starts, M_cap = _groups(c, seed)
        c.update(sizes=sizes, starts=starts, M_cap=M_cap)
        c["split"] = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        c["padded"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        out = dict(dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")
    if c["kind"] == "gemm":
        E, N, K = c["E"], c["N"], c["K"]
        c["a"], c["a_s"] = _quantize_rows(_rows(g, c, sizes, starts, M_cap, K))
        c["b"] = torch.empty(E, N, K, dtype=F8, device="cuda")
        c["b_s"] = torch.empty(E, -(-N // BLOCK), -(-K // BLOCK), dtype=torch.float32, device="cuda")
        for e in range(E):
            w = 0.02 * _randn(g, N, K) * torch.exp(0.3 * _randn(g, N, 1))
            c["b"][e], c["b_s"][e] = _quantize_tiles(w.to(torch.bfloat16))
        c["c"] = torch.zeros(M_cap, N, **out)   # rows that belong to no group are not written: they stay zero
        return c
    if c["kind"] == "wgrad":
        P, Q = c["P"], c["Q"]
        for name, width, size in (("a", P, 1e-3), ("b", Q, 1.0)):
            x = _rows(g, c, sizes, starts, M_cap, width).float() * size
            c[name], c[name + "_s"] = _quantize_rows(x.t().to(torch.bfloat16).contiguous())
        c["c"] = torch.empty(c["E"], P, Q, **out)
        return c
    if c["kind"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        logits = _randn(g, T, E) + 1.4 * _randn(g, 1, E)
        c["logits"] = logits
        c["expert_idx"] = logits.topk(k, dim=1).indices.to(torch.int32)
        c["dprobs"] = 1e-3 * _randn(g, T, k)
        keep = torch.rand(T, generator=g, device="cuda") >= c["masked"]
        c["token_mask"] = keep.to(torch.uint8) if c["masked"] else None
        c["coefs"] = (1e-2, 1e-3 if c["z"] else 0.0)
        i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
        c.update(counts=torch.empty(E, **i32), n_tokens=torch.empty(1, **i32), prob_mean=torch.empty(E, **f32), loss=torch.empty(2, **f32),
                 dlogits=torch.empty(T, E, **f32))
        return c
    c["grads"] = []
    for n, t in _clip_sizes(c):
        x = torch.empty(n, dtype=t, device="cuda")
        for o in range(0, n, 1 << 28):
            x[o:o + (1 << 28)] = (1e-2 * _randn(g, min(1 << 28, n - o))).to(t)
        c["grads"].append(x)
    c["scaled"] = [torch.empty_like(x) for x in c["grads"]]
    expected = 1e-2 * math.sqrt(sum(n for n, _ in _clip_sizes(c)))
    c["max_norm"] = (0.3 if c["clipped"] else 4.0) * expected
    c["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
    c["sumsq"] = torch.empty(1, dtype=torch.float64, device="cuda")
    return c


# ------------------------------------------------------------- plain forms --
def _spread(s, dim, n):
    return s.repeat_interleave(BLOCK, dim=dim).narrow(dim, 0, n)


def _plain_quantize(s):
    out = {}
    xs = list(s["x"])
    if s["mode"] == "tile":
        q, sc = zip(*(_quantize_tiles(x, s["pow2"]) for x in xs))
        out["q"], out["s"] = torch.stack(q), torch.stack(sc)
        out["qT"], out["sT"] = out["q"].transpose(1, 2).contiguous(), out["s"].transpose(1, 2).contiguous()
        return out
    q, sc = zip(*(_quantize_rows(x, s["pow2"]) for x in xs))
    out["q"], out["s"] = torch.stack(q), torch.stack(sc)
    if s["mode"] == "both":
        q, sc = zip(*(_quantize_rows(x.t(), s["pow2"]) for x in xs))
        out["qT"], out["sT"] = torch.stack(q), torch.stack(sc)
    return out


def _plain_gemm(s):
    c = torch.zeros_like(s["c"])
    for e, (n, o) in enumerate(zip(s["sizes"], s["starts"])):   # one whole product for each expert that has rows
        if n:
            a = s["a"][o:o + n].float() * _spread(s["a_s"][:, o:o + n].t(), 1, s["K"])
            w = s["b"][e].float() * _spread(_spread(s["b_s"][e], 0, s["N"]), 1, s["K"])
            c[o:o + n] = (a @ w.t()).to(c.dtype)
    return {"c": c}


def _plain_wgrad(s):
    c = torch.zeros_like(s["c"])
    for e, (n, o) in enumerate(zip(s["sizes"], s["starts"])):
        if n:
            m, k0, k1 = _up(n, BLOCK), o // BLOCK, (o + _up(n, BLOCK)) // BLOCK
            a = s["a"][:, o:o + m].float() * _spread(s["a_s"][k0:k1].t(), 1, m)
            b = s["b"][:, o:o + m].float() * _spread(s["b_s"][k0:k1].t(), 1, m)
            c[e] = (a @ b.t()).to(c.dtype)
    return {"c": c}


def _plain_balance(s):
    T, E, k = s["T"], s["E"], s["k"]
    x, idx = s["logits"], s["expert_idx"].long()
    keep = torch.ones(T, device=x.device) if s["token_mask"] is None else s["token_mask"].float()
    m = x.amax(1, keepdim=True)
    ex = torch.exp(x - m)
    z = ex.sum(1, keepdim=True)
    p, lse = ex / z, (m + torch.log(z)).squeeze(1)
    picked = torch.zeros(T, E, device=x.device).scatter_add_(1, idx, keep[:, None].expand(T, k).contiguous())
    counts = picked.sum(0, dtype=torch.float64)
    n = keep.sum(dtype=torch.float64)
    d = n.clamp(min=1)
    mean = (p * keep[:, None]).sum(0, dtype=torch.float64) / d
    balance, zc = s["coefs"]
    loss = torch.stack((balance * E * (counts / (k * d) * mean).sum(), zc * (keep * lse.square()).sum(dtype=torch.float64) / d))
    v = keep[:, None] * (balance * E * counts / (k * d * d)).float()[None, :]
    v = v.scatter_add(1, idx, s["dprobs"])
    zt = keep * (2 * zc / d).float() * lse
    dlogits = p * (v - (p * v).sum(1, keepdim=True) + zt[:, None])
    return {"counts": counts.to(torch.int32), "n_tokens": n.to(torch.int32).view(1), "prob_mean": mean.float(), "loss": loss.float(), "dlogits": dlogits}


def _plain_clip(s):
    total = torch.stack([x.float().square().sum(dtype=torch.float64) for x in s["grads"]]).sum()
    norm = torch.sqrt(total)
    f = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0).float()
    return {"norm": norm.float().view(1), "grads": [(x.float() * f).to(x.dtype) for x in s["grads"]]}


# --------------------------------------------------------- the library's --
def _own(s):
    import moe_grouped_mlp_amd as mg

    if s["kind"] == "quantize":
        mode = {"row": mg.QUANT_ROW, "both": mg.QUANT_BOTH, "tile": mg.QUANT_TILE}[s["mode"]]
        mg.moe_quantize_fp8(mode=mode, batch=s["batch"], rows=s["rows"], cols=s["cols"], x=s["x"], q=s["q"], s=s["s"], qT=s.get("qT"),
                            sT=s.get("sT"), pow2=s["pow2"])
        out = {"q": s["q"].view(F8), "s": s["s"]}
        return out if s["mode"] == "row" else {**out, "qT": s["qT"].view(F8), "sT": s["sT"]}
    if s["kind"] == "gemm":
        size = dict(E=s["E"], N=s["N"], K=s["K"], M_cap=s["M_cap"], max_rows=s["T"])
        if "workspace" not in s:   # kept between calls, as a program keeps it
            s["workspace"] = torch.empty(max(1, mg.moe_grouped_gemm_fp8_workspace_size(**size)), dtype=torch.uint8, device="cuda")
        mg.moe_grouped_gemm_fp8(**size, split_sizes=s["split"], padded_offsets=s["padded"], a=s["a"], a_s=s["a_s"], b=s["b"], b_s=s["b_s"], c=s["c"],
                                c_type=mg.TYPE_F32 if s["out"] == "f32" else mg.TYPE_BF16, workspace=s["workspace"])
        return {"c": s["c"]}
    if s["kind"] == "wgrad":
        mg.moe_grouped_wgrad_fp8(E=s["E"], P=s["P"], Q=s["Q"], M_cap=s["M_cap"], split_sizes=s["split"], padded_offsets=s["padded"], a=s["a"],
                                 a_s=s["a_s"], b=s["b"], b_s=s["b_s"], c=s["c"], c_type=mg.TYPE_F32 if s["out"] == "f32" else mg.TYPE_BF16)
        return {"c": s["c"]}
    if s["kind"] == "balance":
        size = dict(T=s["T"], E=s["E"], k=s["k"])
        if "workspace" not in s:
            s["workspace"] = torch.empty(max(1, mg.moe_router_loss_workspace_size(s["T"], s["E"])), dtype=torch.uint8, device="cuda")
        both = dict(logits=s["logits"], expert_idx=s["expert_idx"], counts=s["counts"], n_tokens=s["n_tokens"], token_mask=s["token_mask"],
                    balance_coef=s["coefs"][0], z_coef=s["coefs"][1])
        mg.moe_router_loss(**size, **both, prob_mean=s["prob_mean"], loss=s["loss"], workspace=s["workspace"])
        mg.moe_router_bwd(**size, **both, dprobs=s["dprobs"], dlogits=s["dlogits"])
        return {n: s[n] for n in ("counts", "n_tokens", "prob_mean", "loss", "dlogits")}
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(1, mg.moe_grad_workspace_size(len(s["grads"]))), dtype=torch.uint8, device="cuda")
    mg.moe_grad_sumsq(tensors=s["grads"], sumsq=s["sumsq"], workspace=s["workspace"])
    mg.moe_grad_clip(tensors=s["grads"], out=s["scaled"], sumsq=s["sumsq"], max_norm=s["max_norm"], norm=s["norm"])
    return {"norm": s["norm"], "grads": s["scaled"]}


def run(state):
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "gemm": _plain_gemm, "wgrad": _plain_wgrad, "balance": _plain_balance, "clip": _plain_clip}[state["kind"]](state)


# ----------------------------------------------------------- in 64 bits --
def _e4m3(y):
    """The nearest E4M3 value of each y (64 bits), ties to the even code: steps of 2^(exponent - 3), 2^-9 below 2^-6."""
    mag = y.abs()
    e = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.sign(y) * (torch.round(mag / step) * step).clamp(max=E4M3_MAX)


def _exact_blocks(x, down, across, pow2):
    """Codes' values and scales of one matrix in blocks of down x across, block by block along the columns."""
    R, K = x.shape
    q = torch.empty(R, K, dtype=torch.float64, device=x.device)
    scales = []
    for k in range(0, K, across):
        v = x[:, k:k + across].double()
        m = v.abs().amax(1).clamp(min=SMALLEST)
        m = torch.stack([p.max() for p in m.split(down)]) if down > 1 else m
        s = torch.exp2(torch.ceil(torch.log2(m / E4M3_MAX))) if pow2 else m / E4M3_MAX
        scales.append(s)
        q[:, k:k + across] = _e4m3(v / (s.repeat_interleave(down)[:R] if down > 1 else s)[:, None])
    return q, torch.stack(scales)


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "quantize":
        if s["batch"] * s["rows"] * s["cols"] > 1 << 31:
            return None
        down = BLOCK if s["mode"] == "tile" else 1
        got = [_exact_blocks(x, down, BLOCK, s["pow2"]) for x in s["x"]]
        out = {"q": torch.stack([q for q, _ in got]), "s": torch.stack([v.t() if s["mode"] == "tile" else v for _, v in got])}
        if s["mode"] == "tile":
            return {**out, "qT": out["q"].transpose(1, 2), "sT": out["s"].transpose(1, 2)}
        if s["mode"] == "both":
            got = [_exact_blocks(x.t(), 1, BLOCK, s["pow2"]) for x in s["x"]]
            out.update(qT=torch.stack([q for q, _ in got]), sT=torch.stack([v for _, v in got]))
        return out
    if s["kind"] == "gemm":
        c = torch.zeros(s["M_cap"], s["N"], dtype=torch.float64, device="cuda")
        at_n = torch.arange(s["N"], device="cuda") // BLOCK
        for e in range(s["E"]):
            rows = slice(s["starts"][e], s["starts"][e] + s["sizes"][e])
            for b, k in enumerate(range(0, s["K"], BLOCK)):
                part = s["a"][rows, k:k + BLOCK].double() @ s["b"][e, :, k:k + BLOCK].double().t()
                c[rows] += part * s["a_s"][b, rows].double()[:, None] * s["b_s"][e, :, b].double()[at_n][None, :]
        return {"c": c}
    if s["kind"] == "wgrad":
        c = torch.zeros(s["E"], s["P"], s["Q"], dtype=torch.float64, device="cuda")
        for e in range(s["E"]):
            for m in range(s["starts"][e], s["starts"][e] + s["sizes"][e], BLOCK):
                part = s["a"][:, m:m + BLOCK].double() @ s["b"][:, m:m + BLOCK].double().t()
                c[e] += part * s["a_s"][m // BLOCK].double()[:, None] * s["b_s"][m // BLOCK].double()[None, :]
        return {"c": c}
    if s["kind"] == "balance":
        keep = torch.ones(s["T"], dtype=torch.bool, device="cuda") if s["token_mask"] is None else s["token_mask"].bool()
        x = s["logits"].double().requires_grad_(True)
        idx, (balance, zc) = s["expert_idx"].long(), s["coefs"]
        lse = torch.logsumexp(x, 1)
        p = torch.exp(x - lse[:, None])
        n = int(keep.sum())
        counts = torch.bincount(idx[keep].reshape(-1), minlength=s["E"])
        mean = p[keep].sum(0) / max(n, 1)
        loss = torch.stack((balance * s["E"] * (counts.double() / (s["k"] * max(n, 1)) * mean).sum(), zc * lse[keep].square().sum() / max(n, 1)))
        (loss.sum() + (p.gather(1, idx) * s["dprobs"].double()).sum()).backward()
        return {"counts": counts.int(), "n_tokens": torch.tensor([n], dtype=torch.int32), "prob_mean": mean.detach(), "loss": loss.detach(),
                "dlogits": x.grad}
    total = sum(float(part.double().square().sum()) for x in s["grads"] for part in x.split(1 << 27))
    f = min(1.0, s["max_norm"] / (math.sqrt(total) + EPS))
    return {"norm": np.array([math.sqrt(total)]), "grads": [x.double() * f for x in s["grads"]]}
