"""Calls of moe_few, moe_block_norm and the block that are refused on the host, with what is wrong named (CPU)."""

from mixture_experts_layer_counts_amd import router_for, shape_for
from tests.test_few_norm_abi import P, few, lib  # noqa: F401


def test_few_misaligned_bias(lib):  # noqa: F811
    s, r = shape_for(T=4, D=128, I=64, E=8, k=2), router_for()
    for at in (1, 2, 3):
        assert few(lib, s, router=r, bias=P(4096 + at)) == -1, at
