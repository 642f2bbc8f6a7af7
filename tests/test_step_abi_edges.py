"""More host-side checks of the step's entry points (no GPU needed)."""

import pytest

import torch

import moe_grouped_mlp_amd as m
from moe_grouped_mlp_amd import binding as B

from .test_abi import DEVICE, INVALID, no_device
from .test_step_abi import _refuses, gemm, quant, wgrad


def test_fp8_sums_are_of_bf16_outputs():
    for fn, make in (("moe_grouped_gemm_fp8", gemm), ("moe_grouped_wgrad_fp8", wgrad)):
        _refuses(fn, make, [dict(fp8_sums=1, c_type=m.TYPE_F32)], INVALID)


@no_device
def test_fp8_sums_accepted():
    for fn, make in (("moe_grouped_gemm_fp8", gemm), ("moe_grouped_wgrad_fp8", wgrad)):
        _refuses(fn, make, [dict(fp8_sums=1, c_type=m.TYPE_BF16)], DEVICE)


@no_device
def test_fp8_sums_are_of_the_fp8_layer():
    with pytest.raises(ValueError, match="fp8_sums"):
        m.ExpertBlock(4, 128, 128, 16, 2, fp8_sums=True, device="cpu")


NOTHING = dict(x=None, q=None, s=None, qT=None, sT=None)   # what empty tensors have for addresses
MODES = (m.QUANT_ROW, m.QUANT_COL, m.QUANT_BOTH, m.QUANT_TILE)


@no_device
def test_quantize_of_nothing_needs_no_memory():
    for mode in MODES:
        for size in (dict(rows=0), dict(batch=0), dict(rows=0, batch=0)):
            _refuses("moe_quantize_fp8", quant, [dict(mode=mode, **size, **NOTHING)], DEVICE)


def test_quantize_of_nothing_still_checks_the_sizes():
    _refuses("moe_quantize_fp8", quant, [
        dict(rows=0, cols=40, **NOTHING), dict(rows=0, mode=4, **NOTHING), dict(batch=0, rows=-16, **NOTHING),
        dict(batch=0, rows=24, **NOTHING), dict(rows=0, x_stride=4, **NOTHING), NOTHING], INVALID)


@no_device
def test_quantize_takes_empty_tensors():
    """From Python: the refusal left is that there is no device."""
    import unittest.mock as mock
    u8, bf = torch.empty(0, 48, dtype=torch.uint8), torch.empty(0, 48, dtype=torch.bfloat16)
    f32 = torch.empty(1, 0)
    assert bf.data_ptr() == 0
    with mock.patch.object(B, "_device", lambda: (B._setup(), -1)[1]):   # -1: the CPU tensors' device
        for mode in MODES:
            with pytest.raises(m.MoeError) as e:
                m.moe_quantize_fp8(mode=mode, batch=1, rows=0, cols=48, x=bf, q=u8, s=f32, qT=u8, sT=f32, stream=0)
            assert e.value.status == DEVICE
