"""More host-side checks of the step's entry points (no GPU needed)."""

import pytest

import moe_grouped_mlp_amd as m

from .test_abi import DEVICE, INVALID, no_device
from .test_step_abi import _refuses, gemm, wgrad


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
