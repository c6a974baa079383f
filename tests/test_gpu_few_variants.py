"""moe_few where test_gpu_few.py does not go: every kernel that the launcher chooses between, with K long enough that
each wave refills its stages and runs its steady loop, draws of several items, and a router in several K parts. The
comments name what run_few's rule makes of a case (grid: 512 workgroups).

bf16: the bounds of test_gpu_few.py.

MXFP8, with long K: an error per token, of its RMS over the D outputs. The matrix core's sums of 8-bit products are
up to 2^-12 of a large product off, so 2^-9 of the values of h fall on the other side of a border between two values
of E4M3, each by a step, at most 2^-3 of itself: RMS(dh) <= 2^-3 sqrt(2^-9) = 2^-7.5 of h's, over many tokens. In
one token a single value far above the RMS may be among them, and a block of 32 whose largest value lies at a power
of two may take the next one: values of one block B then move by at most 2^-3 of themselves (the largest where it is
cut off at 448 or not), ||dh|| <= 2^-3 ||h_B||. Such a block is one in 2^9 or so, and a token's expert has 2^6 or
2^7 of them: one is to be expected here and there, two at the block of the largest values are not. w_down's entries
are independent of dh and of h, of one size: an expert's output y moves by RMS(dy) / RMS(y) = ||dh|| / ||h||, to a
few percent (D >= 2048 outputs). So a token's error is at most 1.25 sum_s g_s RMS(y_s) (2^-7 + 2^-3 max_B ||h_B|| /
||h||) over its experts, and the shared expert as one of gate 1. A stage of K read from a wrong place, one of n,
changes h by sqrt(2 / n), 0.18 of it or more.
"""

import pytest
import torch

from mixture_experts_layer_counts_amd import MoELayer, router_for, shape_for
from tests._gpu import need_gpu, say
from tests.test_gpu_few import U, Case, mx_round, mx_values

pytestmark = pytest.mark.gpu


def ffn(c, x, pre, e, prec):
    """An expert's output of rows in fp64, and the share of its largest block of h."""
    def mat(n):
        v = c.value[pre + n]
        if prec == "bf16":
            return (v if e is None else v[e]).double()
        return mx_values(v[0], v[1]) if e is None else mx_values(v[0][e], v[1][e])
    q = mx_round if prec == "mxfp8" else (lambda v: v)
    a, u = q(x) @ mat("gate").T, q(x) @ mat("up").T
    h = a / (1 + torch.exp(-a)) * u
    blocks = h.unflatten(-1, (-1, 32)).square().sum(-1)
    share = (blocks.amax(-1) / blocks.sum(-1)).sqrt() if prec == "mxfp8" else None
    return q(h) @ mat("down").T, share


def rms(v):
    return v.square().mean(-1).sqrt()


def check_mx(c, r, kw):
    x, w = c.x.double(), c.w_router.double()
    assert bool(((r["logits"].double() - x @ w.T).abs() <= c.D * U * (x.abs() @ w.abs().T)).all())
    _, idx, gate = c.layer.route(None, None, r["logits"], router=router_for(**kw))
    assert torch.equal(idx, r["idx"]) and torch.equal(gate, r["gate"])

    def bound(y, share):
        return rms(y) * (2.0 ** -7 + 2.0 ** -3 * share if share is not None else 2.0 ** -12)
    want, share = ffn(c, x, "s", None, c.sprec)
    tol = bound(want, share)
    for e in torch.unique(idx).tolist():
        t, s = torch.nonzero(idx == e, as_tuple=True)
        y, share = ffn(c, x[t], "", e, c.prec)
        g = gate[t, s].double()
        want[t] += g[:, None] * y
        tol[t] += g * bound(y, share)
    err = rms(r["out32"].double() - want)
    say("  worst token: error / RMS", float((err / rms(want)).max()), "of the bound", float((err / (1.25 * tol)).max()))
    assert bool((err <= 1.25 * tol).all())
    assert torch.equal(r["out"], r["out32"].to(torch.bfloat16))
    assert c.layer.device_error() == 0


def check(T, D, I, E, k, Is, prec, sprec, tiled, router=None):
    dev = need_gpu()
    say("few", T, D, I, E, k, Is, prec, sprec, tiled, router)
    c = Case(dev, T, D, I, E, k, Is, prec, sprec, tiled, seed=T + D + I)
    r = c.layer.few(c.x, c.w_router, c.weights, router=router_for(**router) if router else None)
    kw = router or dict(score="softmax")
    if "mxfp8" in (prec, sprec):
        check_mx(c, r, kw)
    else:
        c.check(r, None, **kw)
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


# (precision, shared precision) of the four kinds of kernel
KINDS = [("bf16", "bf16"), ("bf16", "mxfp8"), ("mxfp8", "bf16"), ("mxfp8", "mxfp8")]
LONG_K = [  # T, D, I, E, k, Is: stages of 64 (bf16) or 128 values, shared out among four waves
    # 16-row up/gate items (576 and 1024 of them): four stages in flight, 8 to 32 of a wave
    (1, 8192, 1024, 9, 8, 2048),
    (1, 4096, 2048, 8, 7, 2048),
    # 64-row down items (768 of 32 rows would be more than a round): 4 to 8 stages of a wave, two in flight
    (1, 8192, 2048, 2, 2, 2048),
    (4, 8192, 2048, 2, 1, 4096),
    # 32-row items, one block of tokens
    (16, 2048, 2048, 64, 6, 2048),
    # 32-row items, up to four blocks of tokens
    (17, 4096, 2048, 5, 2, 2048),
    (64, 2048, 2048, 12, 3, 2048),
]


@pytest.mark.parametrize("prec,sprec", KINDS)
@pytest.mark.parametrize("T,D,I,E,k,Is", LONG_K)
def test_long_k(T, D, I, E, k, Is, prec, sprec):
    check(T, D, I, E, k, Is, prec, sprec, tiled=(T + E) % 2 == 1)


BATCHES = [  # draws of several items
    (64, 512, 640, 128, 8, 640, "bf16", "bf16", False, None),                                    # up/gate
    (64, 2048, 768, 128, 8, 768, "mxfp8", "bf16", True, None),                                   # down, quantising
    (64, 2048, 768, 128, 8, 768, "mxfp8", "mxfp8", False, dict(score="sigmoid", renorm=False)),
    (1, 2048, 768, 128, 8, 768, "mxfp8", "bf16", True, None),
    (1, 2048, 768, 128, 8, 2048, "mxfp8", "mxfp8", False, None),
]


@pytest.mark.parametrize("T,D,I,E,k,Is,prec,sprec,tiled,router", BATCHES)
def test_batches(T, D, I, E, k, Is, prec, sprec, tiled, router):
    check(T, D, I, E, k, Is, prec, sprec, tiled, router)


ENDS = [  # the first and the last of the counters: 65536 columns, 1024 experts
    (2, 65536, 64, 2, 1, 64, "bf16", "bf16", True),
    (20, 65536, 128, 3, 2, 128, "mxfp8", "bf16", False),
    (64, 64, 64, 1024, 16, 65536, "bf16", "bf16", False),
]


@pytest.mark.parametrize("T,D,I,E,k,Is,prec,sprec,tiled", ENDS)
def test_ends_of_the_counters(T, D, I, E, k, Is, prec, sprec, tiled):
    c, r = check(T, D, I, E, k, Is, prec, sprec, tiled)
    # every counter is cleared again: the next call, of another shape, on the same workspace
    other = Case(c.dev, 5, 192, 64, 30, 4, seed=1)
    want = other.layer.few(other.x, other.w_router, other.weights)
    other.layer.ws, other.layer.ws_bytes = c.layer.ws, c.layer.ws_bytes
    got = other.layer.few(other.x, other.w_router, other.weights)
    assert all(torch.equal(got[n], want[n]) for n in got)
    assert other.layer.device_error() == 0
