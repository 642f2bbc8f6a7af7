"""The router's choice, AdamW and the 8-bit integer calls on buffers of more than
2^31 elements: a small input repeated, so that every copy's results are the small
call's, bit for bit."""

import gc

import pytest
import torch

import moe_grouped_mlp_amd as mg

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """Tests after these measure what torch's allocator holds."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def _same(big, small):
    """big is small, several times, along the first axis."""
    n = small.shape[0]
    assert big.shape[0] % n == 0
    return all(torch.equal(big[i:i + n], small) for i in range(0, big.shape[0], n))


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gate_and_gradient(sigmoid):
    E, k, n, times = 256, 8, 1 << 20, 9
    g = torch.Generator(DEV).manual_seed(1)
    logits = torch.randn(n, E, generator=g, device=DEV)
    dprobs = torch.randn(n, k, generator=g, device=DEV)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    kw = dict(E=E, k=k, score=mg.SCORE_SIGMOID if sigmoid else mg.SCORE_SOFTMAX)
    res = []
    for t in (1, times):
        x, d = logits.repeat(t, 1), dprobs.repeat(t, 1)
        assert t == 1 or x.numel() > 2 ** 31
        idx, w = torch.empty(n * t, k, dtype=torch.int32, device=DEV), torch.empty(n * t, k, device=DEV)
        counts = torch.zeros(E, dtype=torch.int32, device=DEV)
        mg.moe_router_gate(T=n * t, logits=x, expert_idx=idx, probs=w, bias=bias, n_groups=8, topk_groups=3, group_top=2, counts=counts, **kw)
        mg.moe_router_gate_bwd(T=n * t, logits=x, expert_idx=idx, dprobs=d, dlogits=x, **kw)
        res.append((idx, w, x, counts))
    for i in range(3):
        assert _same(res[1][i], res[0][i])
    assert torch.equal(res[1][3], res[0][3] * times)


def test_quantize():
    n, cols, times = 4096, 4096, 129
    x = torch.randn(n, cols, generator=torch.Generator(DEV).manual_seed(2), device=DEV).bfloat16()
    res = []
    for t in (1, times):
        y = x.repeat(t, 1)
        assert t == 1 or y.numel() > 2 ** 31
        q, s = torch.empty(n * t, cols, dtype=torch.int8, device=DEV), torch.empty(n * t, device=DEV)
        mg.moe_quantize_int8(rows=n * t, cols=cols, x=y, q=q, s=s)
        res.append((q, s))
    assert _same(res[1][0], res[0][0]) and _same(res[1][1], res[0][1])


def _product(sizes, N, K, a, a_s, b, b_s, out, **kw):
    starts = [0]
    for s in sizes:
        starts.append(starts[-1] + s)
    split, at = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (sizes, starts))
    c = torch.empty(starts[-1], N, dtype=out, device=DEV)
    mg.moe_grouped_gemm_int8(E=len(sizes), N=N, K=K, M_cap=starts[-1], split_sizes=split, padded_offsets=at, a=a, a_s=a_s, b=b, b_s=b_s, c=c,
                             c_type=mg.TYPE_F32 if out == torch.float32 else mg.TYPE_BF16, **kw)
    return c


def test_product_of_many_rows():
    n, N, K, times = 2048, 8208, 8192, 129
    g = torch.Generator(DEV).manual_seed(3)
    a = torch.randint(-127, 128, (n, K), generator=g, device=DEV, dtype=torch.int8)
    b = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    a_s, b_s = torch.rand(n, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    small = _product([n], N, K, a, a_s, b, b_s, torch.bfloat16)
    need = mg.moe_grouped_gemm_int8_workspace_size(1, N, K, n * times)
    big = _product([n * times], N, K, a.repeat(times, 1), a_s.repeat(times), b, b_s, torch.bfloat16,
                   workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    assert n * times * K > 2 ** 31 and big.numel() > 2 ** 31
    assert _same(big, small)


@pytest.mark.parametrize("hint", [0, 16])
def test_product_of_large_weights(hint):
    """hint 16: the kernel for few rows."""
    rows, N, K, E = 3, 8192, 8192, 40
    g = torch.Generator(DEV).manual_seed(4)
    a = torch.randint(-127, 128, (rows, K), generator=g, device=DEV, dtype=torch.int8)
    b = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    a_s, b_s = torch.rand(rows, generator=g, device=DEV), torch.rand(N, generator=g, device=DEV)
    small = _product([rows], N, K, a, a_s, b, b_s, torch.float32)
    assert E * N * K > 2 ** 31
    big = _product([rows] * E, N, K, a.repeat(E, 1), a_s.repeat(E), b.repeat(E, 1), b_s.repeat(E), torch.float32, max_rows=hint)
    assert _same(big, small)


@pytest.mark.parametrize("fp8", [False, True])
def test_adamw(fp8):
    n, times, tail = 1 << 20, 2049, 100
    g = torch.Generator(DEV).manual_seed(5)
    p, d = (torch.randn(n, generator=g, device=DEV).bfloat16() for _ in range(2))
    res = []
    for t in (1, times):
        param, grad = torch.cat([p.repeat(t), p[:tail]]), torch.cat([d.repeat(t), d[:tail]])
        size = param.numel()
        assert t == 1 or size > 2 ** 31
        m, v = (torch.zeros(size, dtype=torch.uint8 if fp8 else torch.float32, device=DEV) for _ in range(2))
        scales = dict(zip(("m_scale", "v_scale"), ([torch.zeros(-(-size // 128), device=DEV)] for _ in range(2)))) if fp8 else {}
        for step in (1, 2):
            mg.moe_adamw(params=[param], grads=[grad], m=[m], v=[v], lr=0.01, step=step, weight_decay=0.1, **scales)
        res.append((param, m, v))
    for a, b in zip(*res):
        assert _same(b[:n * times], a[:n]) and torch.equal(b[n * times:], a[n:])
