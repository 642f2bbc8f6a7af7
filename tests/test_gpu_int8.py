"""8-bit integer rows (moe_quantize_int8) and their grouped product
(moe_grouped_gemm_int8) against the oracle.  Codes, scales and sums have one
right value each, and a product's result is two fp32 multiplications of it and
one rounding: everything is compared bit for bit."""

import gc

import numpy as np
import pytest
import torch

import moe_grouped_mlp_amd as mg
from oracle import layer as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _give_back():
    """Tests after these measure what torch's allocator holds."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


DEV = "cuda"


def setup_module(module):
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    mg.lib()


def _quantize(x, rows=None, cols=None, **kw):
    rows, cols = rows if rows is not None else x.shape[0], cols or x.shape[1]
    q = torch.full((rows, cols), 99, dtype=torch.int8, device=DEV)
    s = torch.full((rows,), -1.0, device=DEV)
    mg.moe_quantize_int8(rows=rows, cols=cols, x=x, q=q, s=s, **kw)
    return q, s


def _bf16(rng, rows, cols, spread=1.0):
    return torch.from_numpy((rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal((rows, 1)))).astype(np.float32)).to(DEV).bfloat16()


def _same(got, want):
    np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("rows", [1, 3, 17, 1023, 1030])
@pytest.mark.parametrize("cols", [16, 48, 64, 512, 528, 1040, 2048, 2064, 4096, 4112, 8208])
def test_rows(rows, cols):
    x = _bf16(np.random.default_rng(rows + cols), rows, cols)
    q, s = _quantize(x)
    rq, rs = ol.quantize_int8(x.double().cpu().numpy())
    _same(q, rq)
    _same(s, rs)


@pytest.mark.parametrize("rows,cols", [(3, 16384), (2, 16400), (5, 40000), (1025, 16), (2000, 4112)])
def test_long_rows(rows, cols):
    x = _bf16(np.random.default_rng(cols), rows, cols)
    q, s = _quantize(x)
    rq, rs = ol.quantize_int8(x.double().cpu().numpy())
    _same(q, rq)
    _same(s, rs)


@pytest.mark.parametrize("rows", [9, 1100])
def test_every_magnitude_and_odd_values(rows):
    """All 65536 bf16 patterns, rows of zeros, tiny, huge, infinite and NaN ones,
    and halves, which go to the even code."""
    cols = 64
    x = torch.zeros(rows, cols, device=DEV)
    x[1] = 1e-38
    x[2] = 3e38
    x[3, 7] = float("inf")
    x[4, 63] = float("nan")
    x[5, 0] = -float("inf")
    x[6] = torch.arange(cols, device=DEV) - 31.5
    x[6, 0] = 127.0
    x[7] = -127.0
    x[8, :] = -0.0
    x = x.bfloat16()
    q, s = _quantize(x)
    rq, rs = ol.quantize_int8(x.double().cpu().numpy())
    _same(q, rq)
    _same(s, rs)
    assert torch.isnan(s[3:6]).all() and not q[3:6].any()
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(torch.bfloat16)
    y = bits[torch.isfinite(bits)][: 65024 // 64 * 64].view(-1, 64)
    y = y[torch.randperm(y.shape[0], generator=torch.Generator().manual_seed(1)).to(DEV)]
    q, s = _quantize(y)
    rq, rs = ol.quantize_int8(y.double().cpu().numpy())
    _same(q, rq)
    _same(s, rs)


def test_strides_and_row_end():
    x = _bf16(np.random.default_rng(3), 40, 64)
    want = _quantize(x)
    wide = torch.full((40, 72), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :64] = x
    got = _quantize(wide.view(-1), rows=40, cols=64, x_stride=72)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for end in (-5, 0, 1, 17, 40, 1000):
        q, s = _quantize(x, row_end=torch.tensor([end], dtype=torch.int32, device=DEV))
        n = min(max(end, 0), 40)
        assert torch.equal(q[:n], want[0][:n]) and (q[n:] == 99).all() and torch.equal(s[:n], want[1][:n]) and (s[n:] == -1).all()


def test_nothing():
    e = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    _quantize(e, rows=0, cols=16)
    torch.cuda.synchronize()


# ----------------------------------------------------------------- product --
def _starts(sizes, align=128):
    s = [0]
    for n in sizes:
        s.append(s[-1] + -(-n // align) * align)
    return s


def _operands(rng, E, M, N, K):
    a, b = rng.integers(-127, 128, (M, K)).astype(np.int8), rng.integers(-127, 128, (E, N, K)).astype(np.int8)
    return a, np.exp(rng.standard_normal(M)).astype(np.float32), b, np.exp(rng.standard_normal((E, N))).astype(np.float32)


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _product(a, a_s, b, b_s, sizes, starts, out=torch.bfloat16, workspace=None, ldc=0, **kw):
    E, N, K = b.shape
    M = a.shape[0]
    c = torch.full((M, ldc or N), -3.0, dtype=out, device=DEV)
    need = mg.moe_grouped_gemm_int8_workspace_size(E, N, K, M, kw.get("max_rows", 0))
    if workspace is None:
        workspace = torch.full((max(1, need),), 0xFF, dtype=torch.uint8, device=DEV)
    mg.moe_grouped_gemm_int8(E=E, N=N, K=K, M_cap=M, split_sizes=_dev(np.array(sizes, np.int32)), padded_offsets=_dev(np.array(starts, np.int32)),
                             a=_dev(a), a_s=_dev(a_s), b=_dev(b), b_s=_dev(b_s), c=c, ldc=ldc,
                             c_type=mg.TYPE_F32 if out == torch.float32 else mg.TYPE_BF16, workspace=workspace, **kw)
    return c


def _check_product(ops, sizes, starts, out=torch.bfloat16, **kw):
    ref = ol.product_int8(*ops, sizes, starts, ops[0].shape[0])
    got = _product(*ops, sizes, starts, out=out, **kw)
    want = _dev(ref).to(out)   # (torch rounds to nearest even)
    inside = ~torch.isnan(_dev(ref))
    N = ops[2].shape[1]
    assert torch.equal(got[:, :N][inside], want[inside])
    assert (got[:, :N][~inside] == -3.0).all() and (got[:, N:] == -3.0).all()


CASES = [([1], 16, 16), ([2, 0, 3], 48, 144), ([17, 1, 0, 30], 272, 112), ([33, 70], 256, 128), ([64, 65, 128, 129], 512, 256), ([200, 7], 1040, 400),
         ([256, 300, 0, 513], 336, 1168), ([5, 260, 64], 272, 2064), ([1000], 784, 640)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_product(case, out):
    sizes, N, K = case
    starts = _starts(sizes)
    ops = _operands(np.random.default_rng(N + K), len(sizes), starts[-1] + 64, N, K)
    _check_product(ops, sizes, starts, out)
    _check_product(ops, sizes, starts, out, max_rows=max(sizes))
    packed = _starts(sizes, 1)   # groups that start at any row
    _check_product(ops, sizes, packed, out)


@pytest.mark.parametrize("hint", [1, 5, 16, 17, 32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_few_rows(hint, out):
    """The kernel for few rows, with groups larger than was said, too."""
    sizes = [3, 0, 16, 1, 40]
    starts = _starts(sizes)
    for N, K in ((16, 16), (144, 528), (272, 4112), (48, 2032)):
        ops = _operands(np.random.default_rng(N), 5, starts[-1], N, K)
        _check_product(ops, sizes, starts, out, max_rows=hint)


@pytest.mark.parametrize("case", [([100, 100], 112, 4736), ([200, 1], 512, 8192), ([300], 272, 8208), ([64, 0, 64], 48, 16384)], ids=str)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_cut_along_k(case, out):
    sizes, N, K = case
    starts = _starts(sizes)
    ops = _operands(np.random.default_rng(K), len(sizes), starts[-1], N, K)
    assert mg.moe_grouped_gemm_int8_workspace_size(len(sizes), N, K, starts[-1]) > 0
    _check_product(ops, sizes, starts, out)
    one = torch.empty(1, dtype=torch.uint8, device=DEV)   # too small: not cut, and the same bits
    assert torch.equal(_product(*ops, sizes, starts, out=out), _product(*ops, sizes, starts, out=out, workspace=one))


def test_many_tiles():
    """More tiles than CUs, of every height, in every tile size."""
    rng = np.random.default_rng(5)
    sizes = [int(v) for v in rng.integers(0, 900, 20)]
    starts = _starts(sizes)
    for N, K in ((1040, 272), (3600, 144)):
        ops = _operands(rng, 20, starts[-1], N, K)
        for out in (torch.bfloat16, torch.float32):
            _check_product(ops, sizes, starts, out)


@pytest.mark.parametrize("rows,N,K,out", [(4352, 4096, 4112, torch.bfloat16), (4400, 4096, 4112, torch.float32), (8000, 2304, 4128, torch.bfloat16)])
def test_last_round_cut_along_k(rows, N, K, out):
    """More tiles than CUs, and a last round of a few, which are cut."""
    g = torch.Generator(DEV).manual_seed(rows)
    sizes = [rows - 300, 0, 300]
    starts = _starts(sizes)
    a = torch.randint(-127, 128, (starts[-1], K), generator=g, device=DEV, dtype=torch.int8)
    b = torch.randint(-127, 128, (3, N, K), generator=g, device=DEV, dtype=torch.int8)
    a_s, b_s = torch.rand(starts[-1], generator=g, device=DEV), torch.rand(3, N, generator=g, device=DEV)
    got = {}
    need = mg.moe_grouped_gemm_int8_workspace_size(3, N, K, starts[-1])
    assert need > 0
    for ws in (None, torch.empty(need, dtype=torch.uint8, device=DEV)):
        c = torch.full((starts[-1], N), -3.0, dtype=out, device=DEV)
        mg.moe_grouped_gemm_int8(E=3, N=N, K=K, M_cap=starts[-1], split_sizes=_dev(np.array(sizes, np.int32)), padded_offsets=_dev(np.array(starts, np.int32)),
                                 a=a, a_s=a_s, b=b, b_s=b_s, c=c, c_type=mg.TYPE_F32 if out == torch.float32 else mg.TYPE_BF16, workspace=ws)
        for e, (n, o) in enumerate(zip(sizes, starts)):
            s = (a[o:o + n].double() @ b[e].double().t().contiguous()).float()   # (sums below 2^53 are exact)
            assert torch.equal(c[o:o + n], (s * a_s[o:o + n, None] * b_s[e][None, :]).to(out))
            assert (c[o + n:starts[e + 1]] == -3.0).all()
        got[ws is None] = c
    assert torch.equal(got[True], got[False])


def test_extremes_do_not_overflow():
    """The longest K with the largest codes, either sign."""
    K = 131056
    a, b = np.full((40, K), -128, np.int8), np.full((1, 16, K), -128, np.int8)
    b[0, 8:] = 127
    ones = np.ones(40, np.float32), np.ones((1, 16), np.float32)
    for rows in (16, 40):
        _check_product((a, ones[0], b, ones[1]), [rows], [0, 128], torch.float32, max_rows=rows)


def test_scales_that_are_not_finite_stay_in_their_rows():
    sizes, N, K = [40, 3], 64, 128
    starts = _starts(sizes)
    a, a_s, b, b_s = _operands(np.random.default_rng(1), 2, starts[-1], N, K)
    a_s[5], b_s[0, 7], a[6] = np.nan, np.inf, 0
    for kw in (dict(), dict(max_rows=16)):
        c = _product(a, a_s, b, b_s, sizes, starts, torch.float32, **kw).cpu().numpy()
        ref = ol.product_int8(a, a_s, b, b_s, sizes, starts, starts[-1])
        at = np.zeros(len(ref), bool)
        for n, o in zip(sizes, starts):
            at[o:o + n] = True
        np.testing.assert_array_equal(c[at], ref[at])


def test_strides_margin_and_offsets():
    sizes, N, K = [30, 70], 48, 144
    starts = _starts(sizes)
    ops = _operands(np.random.default_rng(2), 2, starts[-1], N, K)
    _check_product(ops, sizes, starts, ldc=56)
    _check_product(ops, sizes, starts, torch.float32, ldc=64)
    cu = torch.cuda.get_device_properties(0).multi_processor_count
    _check_product(ops, sizes, starts, cu_margin=cu - 3)
    _check_product(ops, sizes, starts, cu_margin=cu - 3, max_rows=16)
    # experts apart in memory
    a, a_s, b, b_s = ops
    bw, sw = np.full((2, N * K + 32), 55, np.int8), np.full((2, N + 3), np.nan, np.float32)
    bw[:, :N * K], sw[:, :N] = b.reshape(2, -1), b_s
    c = torch.full((starts[-1], N), -3.0, dtype=torch.bfloat16, device=DEV)
    mg.moe_grouped_gemm_int8(E=2, N=N, K=K, M_cap=starts[-1], split_sizes=_dev(np.array(sizes, np.int32)), padded_offsets=_dev(np.array(starts, np.int32)),
                             a=_dev(a), a_s=_dev(a_s), b=_dev(bw), b_s=_dev(sw), c=c, b_stride=N * K + 32, b_s_stride=N + 3)
    assert torch.equal(c, _product(*ops, sizes, starts))
    # groups that run past the next one's start or the buffer are cut
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _product(*ops, [200, 300], starts, err_flag=err)
    assert err.item() == mg.DEVERR_BAD_OFFSETS
    assert torch.equal(got, _product(*ops, [128, 128], starts))


def test_captured_with_another_stream():
    sizes, N, K = [100, 100], 112, 4736
    starts = _starts(sizes)
    rng = np.random.default_rng(3)
    x = _bf16(rng, starts[-1], K)
    b, b_s = _quantize(_bf16(rng, 2 * N, K))
    split, pad = _dev(np.array(sizes, np.int32)), _dev(np.array(starts, np.int32))
    need = mg.moe_grouped_gemm_int8_workspace_size(2, N, K, starts[-1])

    def run(x, q, s, c, ws, stream=None):
        mg.moe_quantize_int8(rows=starts[-1], cols=K, x=x, q=q, s=s, row_end=pad[2:], stream=stream)
        mg.moe_grouped_gemm_int8(E=2, N=N, K=K, M_cap=starts[-1], split_sizes=split, padded_offsets=pad, a=q, a_s=s, b=b, b_s=b_s, c=c, workspace=ws, stream=stream)

    def bufs():
        return (torch.empty(starts[-1], K, dtype=torch.int8, device=DEV), torch.empty(starts[-1], device=DEV),
                torch.zeros(starts[-1], N, dtype=torch.bfloat16, device=DEV), torch.empty(need, dtype=torch.uint8, device=DEV))
    held, mine = bufs(), bufs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(x, *held)
    side = torch.cuda.Stream()
    for seed in range(4):
        y = _bf16(np.random.default_rng(seed), starts[-1], K)
        x.copy_(y)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        run(y, *mine, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(held[2], mine[2]) and torch.equal(held[0], mine[0])


def test_refusals():
    x, q, s = torch.zeros(4, 32, dtype=torch.bfloat16, device=DEV), torch.zeros(4, 32, dtype=torch.int8, device=DEV), torch.zeros(4, device=DEV)
    ok = dict(rows=4, cols=32, x=x, q=q, s=s)
    for bad in (dict(x=x.float()), dict(q=q.view(torch.uint8)), dict(s=s[:3]), dict(rows=5), dict(x=x.t()), dict(x_stride=40), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            mg.moe_quantize_int8(**{**ok, **bad})
    with pytest.raises(mg.MoeError):
        mg.moe_quantize_int8(**{**ok, "cols": 24})
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    two = torch.zeros(2, dtype=torch.int32, device=DEV)
    ok = dict(E=1, N=16, K=32, M_cap=4, split_sizes=one, padded_offsets=two, a=q, a_s=s, b=torch.zeros(1, 16, 32, dtype=torch.int8, device=DEV),
              b_s=torch.zeros(1, 16, device=DEV), c=torch.zeros(4, 16, dtype=torch.bfloat16, device=DEV))
    mg.moe_grouped_gemm_int8(**ok)
    for bad in (dict(a=q.view(torch.uint8)), dict(b=q), dict(a_s=s[:3]), dict(b_s=s), dict(c_type=mg.TYPE_F32), dict(padded_offsets=one),
                dict(workspace=s), dict(ldc=24), dict(M_cap=5)):
        with pytest.raises(ValueError):
            mg.moe_grouped_gemm_int8(**{**ok, **bad})
