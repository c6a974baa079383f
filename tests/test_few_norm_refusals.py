"""Calls of moe_few, moe_block_norm and the block that are refused on the host, with what is wrong named (CPU)."""

import ctypes

import pytest
import torch

from mixture_experts_layer_counts_amd import MoEBackward, block_norm, block_norm_backward, router_for, shape_for
from tests.test_few_norm_abi import BIG, P, backward, few, forward, lib, norm  # noqa: F401


def test_few_misaligned_bias(lib):  # noqa: F811
    s, r = shape_for(T=4, D=128, I=64, E=8, k=2), router_for()
    for at in (1, 2, 3):
        assert few(lib, s, router=r, bias=P(4096 + at)) == -1, at


def test_dropout_of_everything(lib):  # noqa: F811
    """A probability whose threshold is all of 2^32: no 32-bit word reaches it, and none is below it either way."""
    for p in (1.0 - 2.0 ** -33, 1.0 - 2.0 ** -40, 1.0 - 2.0 ** -53):
        n = norm(dropout=p)
        assert forward(lib, n, rng=P(7 * BIG)) == -1, p
        assert backward(lib, n, rng=P(13 * BIG)) == -1, p
        assert lib.moe_block_norm_backward_workspace_bytes(ctypes.byref(n), ctypes.byref(ctypes.c_size_t())) == -1
    # the largest one there is
    ok = norm(dropout=1.0 - 2.0 ** -32)
    assert lib.moe_block_norm_backward_workspace_bytes(ctypes.byref(ok), ctypes.byref(ctypes.c_size_t())) == 0


def test_streams_that_are_no_tensors(lib):  # noqa: F811
    for v in (None, 1.0, [[0.0] * 8]):
        with pytest.raises(TypeError, match="x must be a tensor"):
            block_norm(v)
        with pytest.raises(TypeError, match="z must be a tensor"):
            block_norm_backward(v, None, None, None)


def test_backward_of_a_block_that_kept_nothing(lib):  # noqa: F811
    x = torch.zeros((4, 64))
    back = MoEBackward(shape_for(T=4, D=64, I=64, E=8, k=2), device="cpu")
    few_results = {n: x for n in ("logits", "idx", "gate", "out", "out32", "h", "z", "h_next")}
    with pytest.raises(ValueError, match="train=True"):
        back.block({}, x, few_results, x, x, None, pre_weight=x[0])
