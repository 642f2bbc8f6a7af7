"""More host-side checks of the router's choice, AdamW and 8-bit integer entry points (no GPU needed)."""

from moe_grouped_mlp_amd import binding as B

from .test_abi import DEVICE, INVALID, UNSUPPORTED, _call, no_device
from .test_layer_abi import _adamw, _tensor, bwd, gate
from .test_step_abi import _refuses


def test_the_largest_norm_keeps_64_bits():
    a = B.AdamwArgs()
    a.max_norm = 0.1
    assert a.max_norm == 0.1 and B.AdamwArgs.max_norm.size == 8


def test_adamw_refuses_a_subnormal_eps():
    """0 / eps would not be 0: the reciprocal of a subnormal number is infinite there."""
    for eps in (1e-40, 2.0 ** -127, 1e-300):
        assert _call("moe_adamw", _adamw([_tensor()], eps=eps)) == INVALID, eps


@no_device
def test_adamw_accepts_small_eps():
    for eps in (0.0, 2.0 ** -126, 1e-30):
        assert _call("moe_adamw", _adamw([_tensor()], eps=eps)) == DEVICE, eps


MOST = 2 ** 26 - 16   # tokens of a wave each: whole workgroups of 1024 threads, less than 2^32


def test_tokens_that_a_launch_rounds_up_to_too_many():
    for name, make in (("moe_router_gate", gate), ("moe_router_gate_bwd", bwd)):
        _refuses(name, make, [dict(T=MOST + 1), dict(T=2 ** 26 - 1)], UNSUPPORTED)


@no_device
def test_most_tokens():
    for name, make in (("moe_router_gate", gate), ("moe_router_gate_bwd", bwd)):
        _refuses(name, make, [dict(T=MOST)], DEVICE)
