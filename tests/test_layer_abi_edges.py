"""More host-side checks of the router's choice, AdamW and 8-bit integer entry points (no GPU needed)."""

from moe_grouped_mlp_amd import binding as B


def test_the_largest_norm_keeps_64_bits():
    a = B.AdamwArgs()
    a.max_norm = 0.1
    assert a.max_norm == 0.1 and B.AdamwArgs.max_norm.size == 8
