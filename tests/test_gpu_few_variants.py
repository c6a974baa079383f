"""moe_few where test_gpu_few.py does not go, under its bounds: every kernel that the launcher chooses between, with K
long enough that each wave refills its stages and runs its steady loop, draws of several items, and a router in several
K parts.  The comments name what run_few's rule makes of a case (grid: 512 workgroups)."""

import pytest
import torch

from mixture_experts_layer_counts_amd import MoELayer, router_for, shape_for
from tests._gpu import need_gpu, say
from tests.test_gpu_few import Case

pytestmark = pytest.mark.gpu


def check(T, D, I, E, k, Is, prec, sprec, tiled, router=None):
    dev = need_gpu()
    say("few", T, D, I, E, k, Is, prec, sprec, tiled, router)
    c = Case(dev, T, D, I, E, k, Is, prec, sprec, tiled, seed=T + D + I)
    r = c.layer.few(c.x, c.w_router, c.weights, router=router_for(**router) if router else None)
    c.check(r, None, **(router if router else dict(score="softmax")))
    again = c.layer.few(c.x, c.w_router, c.weights, router=router_for(**router) if router else None)
    assert all(torch.equal(r[n], again[n]) for n in r)
    return c, r


MANY_TOKENS = [  # more than 16 tokens, few experts with long rows: 32-row items, whatever their number
    (17, 4096, 1024, 8, 2, 1024, "bf16", "bf16", True),
    (64, 2048, 1024, 16, 2, 1024, "bf16", "bf16", False),
    (40, 2048, 1024, 8, 2, 1024, "mxfp8", "bf16", True),
]


@pytest.mark.parametrize("T,D,I,E,k,Is,prec,sprec,tiled", MANY_TOKENS)
def test_many_tokens_few_experts(T, D, I, E, k, Is, prec, sprec, tiled):
    c, r = check(T, D, I, E, k, Is, prec, sprec, tiled)
    # one of the tokens alone takes shorter items: the same bits
    one = MoELayer(shape_for(1, D, I, E, k, I_shared=Is, precision=prec, shared_precision=sprec, weights_tiled=tiled),
                   device=c.dev)
    for t in (0, T - 1):
        s = one.few(c.x[t:t + 1].contiguous(), c.w_router, c.weights)
        assert all(torch.equal(r[n][t:t + 1], s[n]) for n in r)
