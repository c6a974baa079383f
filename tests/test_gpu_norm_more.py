"""moe_block_norm and its gradient where test_gpu_norm.py does not go, under its bounds: many gate rows within a run of
rows whose last chunk overlaps, and dropped values in a row that is normalised."""

import pytest
import torch

from mixture_experts_layer_counts_amd import block_norm, block_norm_backward
from tests._gpu import need_gpu, say
from tests.test_gpu_norm import BF, F32, Case, check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,G,wt", [(9000, 41, 9000, F32), (16390, 23, 8195, BF), (9001, 519, 9001, BF)])
def test_many_gate_rows_a_run(T, D, G, wt):
    """A run's part of dw_post is added up group by group, by single values in the chunk that overlaps."""
    dev = need_gpu()
    say("norm, gate rows a run", T, D, G)
    c = Case(dev, T, D, F32, BF, wt, BF, True, G, True, 0.0, seed=T)
    check_forward(c)
    check_backward(c)
