"""The schedule of one rank with at most 1024 routes (one workgroup builds all of
it), against the oracle's Algorithm 1: route counts around the wave and the
workgroup, experts from one to the most there are, every route to one expert,
and ids out of range."""

import numpy as np
import pytest
import torch

from mixture_experts_layer_counts_amd import MoELayer, shape_for
from oracle import moe as ref
from tests._gpu import need_gpu, say

pytestmark = pytest.mark.gpu


def run(dev, routes, T, k, E):
    m = MoELayer(shape_for(T, 128, 64, E, k), device=dev)
    s = m.schedule(torch.from_numpy(routes).to(dev))
    torch.cuda.synchronize()
    return m, {n: v.cpu().numpy() for n, v in s.items()}


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (7, 9, 100), (63, 1, 5), (64, 1, 1024), (65, 1, 64),
                                   (128, 8, 256), (1023, 1, 33), (64, 16, 1024), (1024, 1, 1), (1025, 1, 7)])
@pytest.mark.parametrize("kind", ["random", "one"])
def test_few_routes(T, k, E, kind):
    dev = need_gpu()
    say("schedule few", T, k, E, kind)
    rng = np.random.default_rng(T + E)
    A = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if kind == "random" \
        else np.full((T, k), E - 1, dtype=np.int32)
    m, got = run(dev, A, T, k, E)
    want = ref.schedule(A.reshape(1, T * k), 0, E)
    assert m.device_error() == 0
    for n in ("counts", "offsets", "sched", "route_dst"):
        assert np.array_equal(got[n].ravel(), np.asarray(want[n]).ravel()), n


def test_few_routes_out_of_range():
    dev = need_gpu()
    A = np.array([[0, 9, -1, 3], [3, 8, 0, 0]], dtype=np.int32)
    m, got = run(dev, A, 2, 4, 8)
    assert m.device_error() & 0x1
    assert got["counts"].tolist() == [3, 0, 0, 2, 0, 0, 0, 0] and got["offsets"][-1] == 5
    assert got["route_dst"].ravel().tolist() == [0, -1, -1, 3, 4, -1, 1, 2]
    assert got["sched"][:5].tolist() == [0, 6, 7, 3, 4]
