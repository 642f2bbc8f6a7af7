"""What a layer of experts is measured on from its router's choice to its weights' update and their 8-bit integer form for serving.

Five kinds of case:

* ``gate``: the choice of experts from the router's logits, by softmax or sigmoid scores, with a balance bias and groups, and the picks' weights.
* ``gate_bwd``: the gradient of the logits from that of the picks' weights.
* ``adamw``: one AdamW step over a list of tensors, clipped to a largest norm, with states in 32 or in 8 bits.
* ``quantize``: bf16 rows to 8-bit integers with a scale for each row (a token's activations, or a weight's output channel).
* ``gemm``: the experts' grouped product of such activations and weights, for prompts and for single tokens.

``own`` chooses between the plain form (elementary torch operations) and the library's kernels.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 128               # values that share a scale of an 8-bit optimizer state, and the alignment of a group's first row
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -100    # a block or row whose largest magnitude is below this is scaled as if it were this
F8 = torch.float8_e4m3fn
NORM_EPS = 1e-6           # added to the norm before the division of the clipping factor
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1


def _up(n, m):
    return -(-n // m) * m


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one decoding step of 16 tokens through a router of 256 experts in 8 groups, of which 4 stay: latency
        dict(name="gate decode groups", kind="gate", T=16, E=256, k=8, score="sigmoid", bias=True, groups=8, stay=4, top=2, renorm=True, logits="f32",
             masked=0.0, ruled=0.0),
        # the same router over a padded prompt
        dict(name="gate prompt groups", kind="gate", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, stay=4, top=2, renorm=True, logits="f32",
             masked=0.1, ruled=0.0),
        # the router of 128 experts of a training step, its logits in bf16, four weights that sum to one
        dict(name="gate 128 experts", kind="gate", T=16384, E=128, k=4, score="softmax", bias=False, groups=1, stay=1, top=1, renorm=True, logits="bf16",
             masked=0.0, ruled=0.0),
        # the gradient of a small layer's router: latency
        dict(name="gate_bwd small", kind="gate_bwd", T=256, E=8, k=2, score="softmax", renorm=True, logits="f32", dropped=0.0),
        # the gradient of a layer of 256 experts whose weights are not renormalised: every logit has one
        dict(name="gate_bwd 256 experts", kind="gate_bwd", T=16384, E=256, k=8, score="softmax", renorm=False, logits="f32", dropped=0.1),
        # twelve small parameters of odd sizes (norms, biases, routers), in both types, states in 32 bits
        dict(name="adamw many small", kind="adamw", tensors=12, largest=200_001, dtype="mixed", grad="same", master=False, state="f32", clipped=True,
             stochastic=False),
        # the two stacked weights of 8 wide experts, bf16 with a 32-bit copy, 32-bit gradients and states
        dict(name="adamw expert weights", kind="adamw", tensors=2, largest=8 * 14336 * 4096, dtype="bf16", grad="f32", master=True, state="f32", clipped=True,
             stochastic=False),
        # the same weights trained in bf16 with states of 8 bits
        dict(name="adamw 8-bit states", kind="adamw", tensors=2, largest=8 * 14336 * 4096, dtype="bf16", grad="same", master=False, state="fp8", clipped=True,
             stochastic=True),
        # the hidden vectors of a decoding step: latency
        dict(name="quantize rows decode", kind="quantize", rows=16, cols=4096),
        # the activations between the two products of a long prompt
        dict(name="quantize activations", kind="quantize", rows=17408, cols=14336),
        # one decoding step of 8 tokens, two experts each: two rows for each of 8 experts, the weights' bytes count
        dict(name="gemm decode", kind="gemm", E=8, k=2, T=8, N=28672, K=4096, skew="even", empty=0, out="bf16"),
        # the second product of a prompt through a layer of 8 wide experts
        dict(name="gemm wide experts", kind="gemm", E=8, k=2, T=8192, N=4096, K=14336, skew="biased", empty=0, out="bf16"),
    ]


def _between(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    kind = rng.choice(("gate", "gate", "gate_bwd", "adamw", "quantize", "gemm", "gemm"))
    if kind == "gate":
        groups = rng.choice((1, 1, 2, 4, 8, 16))
        E = groups * _between(rng, max(2, 16 // groups), 1024 // groups)
        stay = rng.randint(1, groups)
        k = rng.randint(1, min(8, E // groups * stay))
        return dict(kind=kind, T=_between(rng, 1, max(1, min(32768, (1 << 22) // E))), E=E, k=k, score=rng.choice(("softmax", "sigmoid")),
                    bias=rng.random() < 0.6, groups=groups, stay=stay, top=rng.choice((1, 2)), renorm=rng.random() < 0.6, logits=rng.choice(("f32", "f32", "bf16")),
                    masked=rng.choice((0.0, 0.1, 0.5)), ruled=rng.choice((0.0, 0.0, 0.2)))
    if kind == "gate_bwd":
        E = _between(rng, 2, 1024)
        return dict(kind=kind, T=_between(rng, 1, max(1, min(32768, (1 << 22) // E))), E=E, k=rng.randint(1, min(8, E)), score=rng.choice(("softmax", "sigmoid")),
                    renorm=rng.random() < 0.5, logits=rng.choice(("f32", "f32", "bf16")), dropped=rng.choice((0.0, 0.1, 0.5)))
    if kind == "adamw":
        state = rng.choice(("f32", "fp8"))
        return dict(kind=kind, tensors=_between(rng, 1, 12), largest=_between(rng, 100, 20_000_000), dtype=rng.choice(("bf16", "f32", "mixed")),
                    grad=rng.choice(("same", "f32")), master=rng.random() < 0.5, state=state, clipped=rng.random() < 0.7,
                    stochastic=state == "fp8" and rng.random() < 0.6)
    if kind == "quantize":
        cols = _between(rng, 16, 16384, 16)
        return dict(kind=kind, rows=_between(rng, 1, min(32768, max(64, (1 << 27) // cols))), cols=cols)
    E = _between(rng, 1, 96)
    k = rng.choice([j for j in (1, 2, 4, 8) if j <= E])
    empty = rng.choice((0, 0, E // 4)) if E - E // 4 >= k else 0
    T = _between(rng, 1, 8192)
    N = _between(rng, 64, 8192, 16)
    K = _between(rng, 64, max(64, min(8192, (1 << 29) // (E * N))), 16)
    T = max(1, min(T, int(6e11 / (k * N * K))))
    return dict(kind=kind, E=E, k=k, T=T, N=N, K=K, skew=rng.choice(("even", "biased", "zipf")), empty=empty, out=rng.choice(("bf16", "f32")))


def _sizes(case):
    """Rows of each expert, largest first: the same for every seed (which expert has which goes by the seed)."""
    E, live, M = case["E"], case["E"] - case["empty"], case["T"] * case["k"]
    at = (np.arange(live) + 0.5) / live
    if case["skew"] == "zipf":
        w = 1.0 / np.arange(1, live + 1) ** 1.2
    elif case["skew"] == "biased":   # loads of a router whose experts' logits have normal offsets
        w = np.exp(0.7 * math.sqrt(2) * torch.erfinv(torch.from_numpy(1 - 2 * at)).numpy())
    else:
        w = np.ones(live)
    n = np.minimum(np.floor(M * w / w.sum()).astype(np.int64), case["T"])
    while n.sum() < M:               # what rounding left (and what a token's one row for an expert cut off)
        free = np.flatnonzero(n < case["T"])[: M - int(n.sum())]
        n[free] += 1
    return [int(v) for v in n] + [0] * (E - live)


def _adamw_list(case):
    """[(elements, parameter type, gradient type)] of a case."""
    r = random.Random(case["tensors"] * 1_000_003 + case["largest"])
    sizes = [case["largest"]]
    while len(sizes) < case["tensors"]:
        sizes.append(case["largest"] // 2 if case["tensors"] == 2 else _between(r, 1, case["largest"]))
    kinds = {"bf16": (torch.bfloat16,), "f32": (torch.float32,), "mixed": (torch.bfloat16, torch.float32)}[case["dtype"]]
    types = [kinds[i % len(kinds)] for i in range(len(sizes))]
    return [(n, t, torch.float32 if case["grad"] == "f32" else t) for n, t in zip(sizes, types)]


def _bytes(t):
    return 2 if t == torch.bfloat16 else 4


def work(case):
    c = case
    if c["kind"] == "gate":
        n = c["T"] * c["E"]
        return dict(bytes=n * (2 if c["logits"] == "bf16" else 4) + 8 * c["T"] * c["k"], flops=10 * n)
    if c["kind"] == "gate_bwd":
        b = 2 if c["logits"] == "bf16" else 4
        read = c["T"] * c["E"] if c["score"] == "softmax" and not c["renorm"] else c["T"] * c["k"]   # all logits, or the picks' alone
        return dict(bytes=b * (read + c["T"] * c["E"]) + 8 * c["T"] * c["k"], flops=5 * c["T"] * c["E"])
    if c["kind"] == "adamw":
        total = 0
        for n, p, g in _adamw_list(c):
            master = 8 if c["master"] and p == torch.bfloat16 else 0
            weight = _bytes(p) if master else 2 * _bytes(p)   # with a 32-bit copy the weight itself is only written
            total += n * (weight + master + _bytes(g) + (16 if c["state"] == "f32" else 4 + 16 / BLOCK))
        return dict(bytes=total, flops=15 * sum(n for n, _, _ in _adamw_list(c)))
    if c["kind"] == "quantize":
        n = c["rows"] * c["cols"]
        return dict(bytes=3 * n + 4 * c["rows"], flops=2 * n)
    sizes = _sizes(c)
    M, live = sum(sizes), sum(n > 0 for n in sizes)
    return dict(bytes=M * (c["K"] + 4) + live * c["N"] * (c["K"] + 4) + M * c["N"] * (4 if c["out"] == "f32" else 2), flops=2 * M * c["N"] * c["K"])


# ------------------------------------------------------------- preparation --
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _filled(g, n, dtype, values):
    """n values of a generator of fp32 pieces, a piece at a time."""
    x = torch.empty(n, dtype=dtype, device="cuda")
    for o in range(0, n, 1 << 28):
        x[o:o + (1 << 28)] = values(min(1 << 28, n - o)).to(dtype)
    return x


def _quantize_rows(x):
    """x [R][K] -> codes int8 [R][K], scales [R] (fp32): code = round(x * (127 / m)), scale = m / 127, both quotients rounded once."""
    v = x.float()
    m = v.abs().amax(1).clamp(min=SMALLEST).double()
    return torch.round(v * (127.0 / m).float()[:, None]).to(torch.int8), (m / 127.0).float()


def _blocks(x):
    """A flat tensor in rows of BLOCK, the last one filled with zeros."""
    n = x.numel()
    if n % BLOCK:
        x = torch.cat([x, torch.zeros(_up(n, BLOCK) - n, dtype=x.dtype, device=x.device)])
    return x.view(-1, BLOCK)


def _encode(x):
    """A flat fp32 tensor -> the values of its codes before rounding (in rows of BLOCK), and its scales."""
    v = _blocks(x)
    m = v.abs().amax(1).clamp(min=SMALLEST).double()
    return v * (E4M3_MAX / m).float()[:, None], (m / E4M3_MAX).float()


def _codes(y, n):
    return y.to(F8).view(-1)[:n].contiguous()


def _logits(g, c):
    x = _randn(g, c["T"], c["E"]) + (1.4 if c["score"] == "softmax" else 0.5) * _randn(g, 1, c["E"])
    return x.to(torch.bfloat16) if c["logits"] == "bf16" else x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    if c["kind"] == "gate":
        T, E, k = c["T"], c["E"], c["k"]
        c["x"] = _logits(g, c)
        if c["ruled"]:   # experts that are out of service, for all tokens
            c["x"][:, torch.rand(E, generator=g, device="cuda") < c["ruled"]] = -math.inf
        c["balance"] = 0.1 * _randn(g, E) if c["bias"] else None
        c["token_mask"] = (torch.rand(T, generator=g, device="cuda") >= c["masked"]).to(torch.uint8) if c["masked"] else None
        c["scale"] = 2.5 if c["score"] == "sigmoid" else 1.0
        c.update(expert_idx=torch.empty(T, k, **i32), probs=torch.empty(T, k, **f32), counts=torch.zeros(E, **i32))
        return c
    if c["kind"] == "gate_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        c["x"] = _logits(g, c)
        idx = c["x"].float().topk(k, dim=1).indices.to(torch.int32)
        idx[torch.rand(T, generator=g, device="cuda") < c["dropped"]] = -1   # tokens of the padding went nowhere
        c["expert_idx"] = idx
        c["dprobs"] = 1e-3 * _randn(g, T, k)
        c["scale"] = 2.5 if c["score"] == "sigmoid" else 1.0
        c["dlogits"] = torch.empty_like(c["x"])
        return c
    if c["kind"] == "adamw":
        for name in ("params", "grads", "m", "v", "master", "m_scale", "v_scale"):
            c[name + "_t"] = []
        for n, p, gt in _adamw_list(c):
            size = math.exp(random.Random(seed + n).uniform(-1, 1))   # gradients of one tensor are larger than another's
            w = _filled(g, n, torch.float32, lambda j: 0.02 * _randn(g, j))
            c["params_t"].append(w.to(p))
            c["master_t"].append(w if c["master"] and p == torch.bfloat16 else None)
            c["grads_t"].append(_filled(g, n, gt, lambda j: 1e-2 * size * _randn(g, j)))
            m = _filled(g, n, torch.float32, lambda j: 2e-3 * size * _randn(g, j))
            v = _filled(g, n, torch.float32, lambda j: (1e-2 * size * torch.exp(0.5 * _randn(g, j))).square())
            if c["state"] == "f32":
                c["m_t"].append(m)
                c["v_t"].append(v)
            else:   # v is kept as its root
                for name, x in (("m", m), ("v", v.sqrt_())):
                    y, s = _encode(x)
                    c[name + "_t"].append(_codes(y, n))
                    c[name + "_scale_t"].append(s)
                    del y
        norm = math.sqrt(sum(float(x.float().square().sum(dtype=torch.float64)) for x in c["grads_t"]))
        c["sumsq"] = torch.full((1,), norm * norm, dtype=torch.float64, device="cuda") if c["clipped"] else None   # from the norm's own call
        c["max_norm"] = 0.7 * norm
        c["decay"] = [DECAY if i % 3 else 0.0 for i in range(c["tensors"])]   # some (norms, biases) have none
        c["step"], c["rounding_seed"] = 1000, seed & 0xffffffff
        return c
    if c["kind"] == "quantize":
        R, K = c["rows"], c["cols"]
        c["x"] = (_randn(g, R, K) * torch.exp(_randn(g, R, 1))).to(torch.bfloat16)
        c["q"] = torch.empty(R, K, dtype=torch.int8, device="cuda")
        c["s"] = torch.empty(R, **f32)
        return c
    sizes = _sizes(c)
    random.Random(seed).shuffle(sizes)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _up(n, BLOCK))
    E, N, K, M_cap = c["E"], c["N"], c["K"], _up(c["T"] * c["k"] + c["E"] * (BLOCK - 1), BLOCK)
    c.update(sizes=sizes, starts=starts, M_cap=M_cap, split=torch.tensor(sizes, **i32), padded=torch.tensor(starts, **i32))
    x = _randn(g, M_cap, K) * torch.exp(0.5 * _randn(g, M_cap, 1)) * torch.exp(0.5 * _randn(g, 1, K))
    for n, o, end in zip(sizes, starts, starts[1:] + [M_cap]):   # rows between groups are zero, as the permutation leaves them
        x[o + n:end] = 0
    c["a"], c["a_s"] = _quantize_rows(x.to(torch.bfloat16))
    c["b"] = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    c["b_s"] = torch.empty(E, N, **f32)
    for e in range(E):
        w = 0.02 * _randn(g, N, K) * torch.exp(0.3 * _randn(g, N, 1))
        c["b"][e], c["b_s"][e] = _quantize_rows(w.to(torch.bfloat16))
    c["c"] = torch.zeros(M_cap, N, dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")   # rows of no group stay zero
    return c


# ------------------------------------------------------------- plain forms --
def _scores(x, score):
    """Scores of the experts; one whose logit is -inf or NaN is ruled out (0)."""
    if score == "sigmoid":
        return torch.where(x > -math.inf, 1 / (1 + torch.exp(-x)), 0)
    x = torch.where(x > -math.inf, x, -math.inf)
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(m > -math.inf, m, 0))
    z = e.sum(1, keepdim=True)
    return e / torch.where(z > 0, z, 1)


def _weights(x, score, s, live, renorm, scale):
    """The picks' weights from their logits x and scores s (live: slots that hold a pick)."""
    if renorm:   # of the scores times a factor that keeps the largest of them in range
        top = torch.where(live, x, -math.inf).amax(1, keepdim=True)
        top = torch.where(top > -math.inf, top, 0)
        s = torch.where(top < 0, torch.exp(x - top) / (1 + torch.exp(x)), 1 / (1 + torch.exp(-x))) if score == "sigmoid" else torch.exp(x - top)
        s = torch.where(live, s, 0)
        z = s.sum(1, keepdim=True)
        s = s / torch.where(z > 0, z, 1)
    return torch.where(live, scale * s, 0)


def _plain_gate(s):
    T, E, k = s["T"], s["E"], s["k"]
    x = s["x"].double()   # choices next to one another decide: 64 bits
    p = _scores(x, s["score"])
    judged = p if s["balance"] is None else p + s["balance"].double()
    choice = x if s["balance"] is None else judged
    out = ~(x > -math.inf)
    if s["token_mask"] is not None:
        out = out | (s["token_mask"] == 0)[:, None]
    choice = torch.where(out, -math.inf, choice)
    if s["groups"] > 1:
        by = (choice if s["top"] == 1 else torch.where(out, -math.inf, judged)).view(T, s["groups"], -1)
        best = by.sort(dim=2, descending=True).values[:, :, :s["top"]]
        value = torch.where(best > -math.inf, best, 0).sum(2)
        value = torch.where(best[:, :, 0] > -math.inf, value, -math.inf)
        stay = torch.zeros(T, s["groups"], dtype=torch.bool, device=x.device)
        stay.scatter_(1, value.sort(dim=1, descending=True, stable=True).indices[:, :s["stay"]], True)
        choice = torch.where(stay.repeat_interleave(E // s["groups"], dim=1), choice, -math.inf)
    best, idx = choice.sort(dim=1, descending=True, stable=True)
    idx, live = idx[:, :k], best[:, :k] > -math.inf
    xf = s["x"].float()
    pf = _scores(xf, s["score"]) if not s["renorm"] else xf
    w = _weights(xf.gather(1, idx), s["score"], pf.gather(1, idx), live, s["renorm"], s["scale"])
    picked = torch.zeros(T, E, dtype=torch.int32, device=x.device).scatter_(1, idx, live.int())
    s["counts"] += picked.sum(0, dtype=torch.int32)
    return {"expert_idx": torch.where(live, idx, -1).int(), "probs": w, "counts": s["counts"]}


def _plain_gate_bwd(s):
    x, live = s["x"].float(), s["expert_idx"] >= 0
    idx = s["expert_idx"].long().clamp(min=0)
    xi, g = x.gather(1, idx), torch.where(live, s["scale"] * s["dprobs"], 0)
    si = _scores(x, s["score"]).gather(1, idx)
    if s["renorm"]:
        w = _weights(xi, s["score"], si, live, True, 1.0)
        d = w * (g - (w * g).sum(1, keepdim=True))
        if s["score"] == "sigmoid":
            d = d / (1 + torch.exp(xi))
    elif s["score"] == "sigmoid":
        d = g * si / (1 + torch.exp(xi))
    else:
        d = g * si
    out = torch.zeros_like(x).scatter_add_(1, idx, torch.where(live, d, 0))
    if s["score"] == "softmax" and not s["renorm"]:
        out = out - _scores(x, "softmax") * (torch.where(live, d, 0)).sum(1, keepdim=True)
    return {"dlogits": out.to(s["dlogits"].dtype)}


def _mix(x):
    """32 bits to 32 bits (an integer, or a tensor of int64): shifts and odd multipliers."""
    x = ((x ^ (x >> 16)) * 0x7feb352d) & 0xffffffff
    x = ((x ^ (x >> 15)) * 0x846ca68b) & 0xffffffff
    return x ^ (x >> 16)


def _random16(s, tensor, n, device):
    """16 random bits for each of n elements, two elements' from one mixed counter."""
    key = _mix((_mix((s["rounding_seed"] + s["step"] * 0x9e3779b9) & 0xffffffff) + tensor) & 0xffffffff)
    i = torch.arange(n, dtype=torch.int64, device=device)
    h = _mix((key + (i >> 1)) & 0xffffffff)
    return torch.where((i & 1) == 1, h >> 16, h & 0xffff)


def _root_codes(s, tensor, r):
    """Codes and scales of v's root: rounded up with a probability of what is left (stochastic) or to nearest, never from above zero to zero."""
    n = r.numel()
    y, sc = _encode(r)
    y = y.view(-1)[:n]
    if s["stochastic"]:
        z = torch.where(y < 2.0 ** -6, y + 2.0 ** -6, y).double()   # next to a border: 64 bits
        step = torch.exp2(torch.floor(torch.log2(z.clamp(min=2.0 ** -6))) - 3)
        z = torch.floor(z / step + _random16(s, tensor, n, r.device) / 65536.0) * step
        q = torch.where(y < 2.0 ** -6, z - 2.0 ** -6, z).clamp(max=E4M3_MAX).float()
    else:
        q = y.to(F8).float()
    return torch.where((y > 0) & (q == 0), 2.0 ** -9, q).to(F8), sc


def _decode(q, sc):
    n = q.numel()
    return (_blocks(q.float()) * sc[:, None]).view(-1)[:n]


def _clip_factor(s):
    if s["sumsq"] is None:
        return 1.0
    return torch.clamp(s["max_norm"] / (torch.sqrt(s["sumsq"]) + NORM_EPS), max=1.0).float()


def _plain_adamw(s):
    f = _clip_factor(s)
    c1, c2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    for i, (p, g) in enumerate(zip(s["params_t"], s["grads_t"])):
        eight, master = s["state"] == "fp8", s["master_t"][i]
        m = _decode(s["m_t"][i], s["m_scale_t"][i]) if eight else s["m_t"][i]
        v = _decode(s["v_t"][i], s["v_scale_t"][i]).square() if eight else s["v_t"][i]
        d = g.float() * f
        m = BETA1 * m + (1 - BETA1) * d
        v = BETA2 * v + (1 - BETA2) * d * d
        r = torch.sqrt(v)
        w = p.float() if master is None else master
        w = w - (LR * s["decay"][i]) * w - (LR / c1) * (m / (r / math.sqrt(c2) + EPS))
        p.copy_(w)
        if master is not None:
            master.copy_(w)
        if eight:
            y, sc = _encode(m)
            s["m_t"][i].copy_(_codes(y, m.numel()))
            s["m_scale_t"][i].copy_(sc)
            q, sc = _root_codes(s, i, r)
            s["v_t"][i].copy_(q)
            s["v_scale_t"][i].copy_(sc)
        else:
            s["m_t"][i].copy_(m)
            s["v_t"][i].copy_(v)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    names = ("params", "master", "m", "v", "m_scale", "v_scale")
    return {n: [x for x in s[n + "_t"] if x is not None] for n in names if any(x is not None for x in s[n + "_t"])}


def _plain_quantize(s):
    q, sc = _quantize_rows(s["x"])
    return {"q": q, "s": sc}


def _plain_gemm(s):
    c = torch.zeros_like(s["c"])
    for e, (n, o) in enumerate(zip(s["sizes"], s["starts"])):   # one whole product for each expert that has rows
        if n:
            y = s["a"][o:o + n].float() @ s["b"][e].float().t()
            c[o:o + n] = (y * s["a_s"][o:o + n, None] * s["b_s"][e][None, :]).to(c.dtype)
    return {"c": c}


# --------------------------------------------------------- the library's --
def _own(s):
    import moe_grouped_mlp_amd as mg

    if s["kind"] in ("gate", "gate_bwd"):
        both = dict(T=s["T"], E=s["E"], k=s["k"], logits=s["x"], expert_idx=s["expert_idx"], renorm=s["renorm"], scale=s["scale"],
                    score=mg.SCORE_SIGMOID if s["score"] == "sigmoid" else mg.SCORE_SOFTMAX)
        if s["kind"] == "gate_bwd":
            mg.moe_router_gate_bwd(**both, dprobs=s["dprobs"], dlogits=s["dlogits"])
            return {"dlogits": s["dlogits"]}
        mg.moe_router_gate(**both, probs=s["probs"], bias=s["balance"], n_groups=s["groups"], topk_groups=s["stay"], group_top=s["top"],
                           token_mask=s["token_mask"], counts=s["counts"])
        return {n: s[n] for n in ("expert_idx", "probs", "counts")}
    if s["kind"] == "adamw":
        eight = s["state"] == "fp8"
        mg.moe_adamw(params=s["params_t"], grads=s["grads_t"], m=s["m_t"], v=s["v_t"], master=s["master_t"], m_scale=s["m_scale_t"] if eight else None,
                     v_scale=s["v_scale_t"] if eight else None, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=s["decay"], step=s["step"],
                     sumsq=s["sumsq"], max_norm=s["max_norm"], stochastic=s["stochastic"], seed=s["rounding_seed"])
        return _adamw_outputs(s)
    if s["kind"] == "quantize":
        mg.moe_quantize_int8(rows=s["rows"], cols=s["cols"], x=s["x"], q=s["q"], s=s["s"])
        return {"q": s["q"], "s": s["s"]}
    size = dict(E=s["E"], N=s["N"], K=s["K"], M_cap=s["M_cap"], max_rows=s["T"])
    if "workspace" not in s:   # kept between calls, as a program keeps it
        s["workspace"] = torch.empty(max(1, mg.moe_grouped_gemm_int8_workspace_size(**size)), dtype=torch.uint8, device="cuda")
    mg.moe_grouped_gemm_int8(**size, split_sizes=s["split"], padded_offsets=s["padded"], a=s["a"], a_s=s["a_s"], b=s["b"], b_s=s["b_s"], c=s["c"],
                             c_type=mg.TYPE_F32 if s["out"] == "f32" else mg.TYPE_BF16, workspace=s["workspace"])
    return {"c": s["c"]}


def run(state):
    if own:
        return _own(state)
    return {"gate": _plain_gate, "gate_bwd": _plain_gate_bwd, "adamw": _plain_adamw, "quantize": _plain_quantize, "gemm": _plain_gemm}[state["kind"]](state)


# ----------------------------------------------------------- in 64 bits --
def _e4m3(y):
    """The nearest E4M3 value of each y (64 bits), ties to the even code: steps of 2^(exponent - 3), 2^-9 below 2^-6."""
    step = _e4m3_step(y.abs())
    return torch.sign(y) * (torch.round(y.abs() / step) * step).clamp(max=E4M3_MAX)


def _e4m3_step(mag):
    return torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)


def _exact_state(x, at, random16=None):
    """Codes' values and scales of a piece of a state that starts at element `at` (a multiple of BLOCK)."""
    rows = _blocks(x)
    s = rows.abs().amax(1).clamp(min=SMALLEST) / E4M3_MAX
    y = (rows / s[:, None]).view(-1)[:x.numel()]
    if random16 is None:
        return _e4m3(y), s
    step = _e4m3_step(y)
    q = (torch.floor(y / step + random16.double() / 65536) * step).clamp(max=E4M3_MAX)
    return torch.where((y > 0) & (q == 0), 2.0 ** -9, q), s


def _exact_adamw(s):
    f = 1.0 if s["sumsq"] is None else min(1.0, s["max_norm"] / (math.sqrt(float(s["sumsq"])) + NORM_EPS))
    out = {n: [] for n in ("params", "master", "m", "v", "m_scale", "v_scale")}
    for i, n in enumerate(x.numel() for x in s["params_t"]):
        got = {name: [] for name in out}
        bits = _random16(s, i, n, "cuda") if s["stochastic"] else None
        for o in range(0, n, 1 << 27):
            part = slice(o, min(n, o + (1 << 27)))
            m, v = s["m_t"][i][part].double(), s["v_t"][i][part].double()
            if s["state"] == "fp8":
                sc = slice(o // BLOCK, _up(part.stop, BLOCK) // BLOCK)
                m = m * s["m_scale_t"][i][sc].double().repeat_interleave(BLOCK)[:m.numel()]
                v = (v * s["v_scale_t"][i][sc].double().repeat_interleave(BLOCK)[:m.numel()]) ** 2
            d = s["grads_t"][i][part].double() * f
            m, v = BETA1 * m + (1 - BETA1) * d, BETA2 * v + (1 - BETA2) * d ** 2
            w = (s["params_t"][i] if s["master_t"][i] is None else s["master_t"][i])[part].double()
            w = w * (1 - LR * s["decay"][i]) - LR * (m / (1 - BETA1 ** s["step"])) / ((v / (1 - BETA2 ** s["step"])).sqrt() + EPS)
            got["params"].append(w)
            if s["master_t"][i] is not None:
                got["master"].append(w)
            if s["state"] == "fp8":
                q, sc = _exact_state(m, o)
                got["m"].append(q)
                got["m_scale"].append(sc)
                q, sc = _exact_state(v.sqrt(), o, bits[part] if s["stochastic"] else None)
                if not s["stochastic"]:
                    q = torch.where((v > 0) & (q == 0), 2.0 ** -9, q)
                got["v"].append(q)
                got["v_scale"].append(sc)
            else:
                got["m"].append(m)
                got["v"].append(v)
        for name, pieces in got.items():
            if pieces:
                out[name].append(torch.cat(pieces) if len(pieces) > 1 else pieces[0])
    return {name: x for name, x in out.items() if x}


def _exact_picks(s):
    """(picks [T][k] with -1, choices' logits in 64 bits), token by token in Python's own terms over numpy arrays."""
    x = s["x"].double().cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        if s["score"] == "sigmoid":
            p = 1 / (1 + np.exp(-x))
        else:
            p = np.exp(x - np.max(x, axis=1, keepdims=True, initial=-1e300))
            p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    judged = p if s["balance"] is None else p + s["balance"].double().cpu().numpy()
    choice = (x if s["balance"] is None else judged).copy()
    gone = ~(x > -math.inf)
    if s["token_mask"] is not None:
        gone |= (s["token_mask"].cpu().numpy() == 0)[:, None]
    choice[gone] = -math.inf
    if s["groups"] > 1:
        by = np.where(gone, -math.inf, choice if s["top"] == 1 else judged).reshape(s["T"], s["groups"], -1)
        best = -np.sort(-by, axis=2)[:, :, :s["top"]]
        value = np.where(best[:, :, 0] > -math.inf, np.where(best > -math.inf, best, 0).sum(2), -math.inf)
        order = np.argsort(-value, axis=1, kind="stable")[:, s["stay"]:]
        grouped = choice.reshape(s["T"], s["groups"], -1)
        np.put_along_axis(grouped, order[:, :, None].repeat(grouped.shape[2], 2), -math.inf, axis=1)
        choice = grouped.reshape(x.shape)
    order = np.argsort(-choice, axis=1, kind="stable")[:, :s["k"]]
    return np.where(np.take_along_axis(choice, order, 1) > -math.inf, order, -1), p


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "gate":
        idx, p = _exact_picks(s)
        w = np.where(idx >= 0, np.take_along_axis(p, np.maximum(idx, 0), 1), 0.0)
        if s["renorm"]:
            w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
        counts = np.bincount(idx[idx >= 0].reshape(-1), minlength=s["E"]).astype(np.int32)
        return {"expert_idx": idx.astype(np.int32), "probs": s["scale"] * w, "counts": counts}
    if s["kind"] == "gate_bwd":
        x = s["x"].double().requires_grad_(True)
        live = s["expert_idx"] >= 0
        p = torch.softmax(x, 1) if s["score"] == "softmax" else torch.sigmoid(x)
        w = p.gather(1, s["expert_idx"].long().clamp(min=0)) * live
        if s["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        (s["scale"] * w * s["dprobs"].double()).sum().backward()
        return {"dlogits": x.grad}
    if s["kind"] == "adamw":
        return _exact_adamw(s)
    if s["kind"] == "quantize":
        m = s["x"].double().abs().amax(1).clamp(min=SMALLEST)
        return {"q": None, "s": m / 127}
    c = torch.zeros(s["M_cap"], s["N"], dtype=torch.float64, device="cuda")
    for e, (n, o) in enumerate(zip(s["sizes"], s["starts"])):
        for r in range(o, o + n, 2048):
            rows = slice(r, min(r + 2048, o + n))
            c[rows] = (s["a"][rows].double() * s["a_s"][rows].double()[:, None]) @ (s["b"][e].double() * s["b_s"][e].double()[:, None]).t()
    return {"c": c}
