"""Routing from scores (moe_route_scored) and its gradient (moe_route_backward)
on the CPU: the oracle against torch's double autograd and differences, and the
host-side checks of the entry points."""

import ctypes
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

from mixture_experts_layer_counts_amd import _lib, router_for, shape_for
from oracle import scored
from tests.test_abi import lib, ws_bytes  # noqa: F401


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_oracle_gradient(kind, renorm):
    rng = np.random.default_rng(3)
    l, dg = rng.standard_normal((7, 12)), rng.standard_normal((7, 3))
    idx = scored.choose(scored.scores(l, kind), rng.standard_normal(12) * 0.1, 3, 4, 2)
    got = scored.backward(l, idx, dg, kind, renorm, 2.5)
    t = torch.tensor(l, requires_grad=True)
    s = torch.sigmoid(t) if kind == "sigmoid" else torch.softmax(t, dim=1)
    w = torch.gather(s, 1, torch.from_numpy(idx).long())
    g = 2.5 * (w / w.sum(1, keepdim=True) if renorm else w)
    (g * torch.from_numpy(dg)).sum().backward()
    assert np.abs(got - t.grad.numpy()).max() < 1e-13

    def loss(v):
        return (scored.gates(scored.scores(v, kind), idx, renorm, 2.5) * dg).sum()
    h = 1e-6
    for t_, e in ((0, int(idx[0, 0])), (3, int(idx[3, 2])), (5, 11)):
        up, dn = l.copy(), l.copy()
        up[t_, e] += h
        dn[t_, e] -= h
        assert abs((loss(up) - loss(dn)) / (2 * h) - got[t_, e]) < 1e-8


def test_oracle_gradient_of_saturated_sigmoids():
    # s (1 - s) = exp(-|l|) / (1 + exp(-|l|))^2 to full precision, against 40 decimal digits
    l = np.array([[-60.0, -37.5, -8.0, 0.25, 20.0, 30.0, 37.5, 60.0]])
    idx, dg = np.arange(8, dtype=np.int32)[None], np.linspace(-1.0, 2.0, 8)[None]
    got = scored.backward(l, idx, dg, "sigmoid", False, 2.5)
    with localcontext() as c:
        c.prec = 40
        for e in range(8):
            z = (-abs(Decimal(l[0, e]))).exp()
            want = Decimal(2.5) * Decimal(dg[0, e]) * z / (1 + z) ** 2
            # two logistic functions and three products, a few 2^-53 each, exp's argument exact
            assert abs(Decimal(got[0, e]) - want) <= Decimal(1e-15) * 2 * abs(want), e


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_oracle_ratios_far_below_the_maximum(kind):
    # two chosen logits one apart: e / (1 + e) and 1 / (1 + e) wherever they lie below 0
    l = np.array([[3.0, -1e4, -10001.0], [3.0, -600.0, -601.0], [0.0, -800.0, -np.inf], [0.0, -np.inf, -np.inf]])
    idx = np.tile(np.array([[1, 2]], dtype=np.int32), (4, 1))
    a = np.e / (1.0 + np.e)
    want = np.array([[a, 1 - a], [a, 1 - a], [1, 0], [0, 0]])
    assert np.abs(scored.ratios(l, idx, kind) - want).max() < 1e-12
    got = scored.backward(l, idx, np.array([[1.0, 3.0]] * 4), kind, True, 2.0)
    # scale p (dg - p . dg): the differences of the two are -2 p_1 and 2 p_0
    dl = 2.0 * a * (1 - a) * 2.0
    assert np.abs(got - np.array([[0, -dl, dl]] * 2 + [[0, 0, 0]] * 2)).max() < 1e-12
    near = np.random.default_rng(1).standard_normal((5, 9))
    ids = scored.choose(scored.scores(near, kind), None, 4)
    gates = scored.gates(scored.scores(near, kind), ids, True, 1.0)
    assert np.abs(scored.ratios(near, ids, kind) - gates).max() < 1e-14


def test_oracle_choice_by_hand():
    s = np.array([[0.9, 0.1, 0.5, 0.45, 0.8, 0.05]])
    # pairs (0.9 0.1) (0.5 0.45) (0.8 0.05): sums 1.0, 0.95, 0.85; maxima 0.9, 0.5, 0.8
    assert scored.choose(s, None, 2, 3, 2, "top2").tolist() == [[0, 2]]
    assert scored.choose(s, None, 2, 3, 2, "max").tolist() == [[0, 4]]
    assert scored.choose(s, np.array([0, 0, 0, 0, 0, 9.0]), 2, 3, 1, "max").tolist() == [[5, 4]]
    assert scored.choose(np.full((1, 4), 0.5), None, 3).tolist() == [[0, 1, 2]]


FAKE = ctypes.c_void_p(4096)  # never dereferenced: every call below returns first


def call(lib, s, r, x=None, w=None, logits=FAKE, idx=FAKE, gate=FAKE):  # noqa: F811
    n = ws_bytes(lib, s)[1]
    return lib.moe_route_scored(ctypes.byref(s), None if r is None else ctypes.byref(r), x, w, None, logits, idx,
                                gate, FAKE, n, None)


def call_backward(lib, s, r, logits=FAKE, idx=FAKE, dgate=FAKE, out=FAKE):  # noqa: F811
    n = ws_bytes(lib, s)[1]
    return lib.moe_route_backward(ctypes.byref(s), None if r is None else ctypes.byref(r), logits, idx, dgate, out,
                                  FAKE, n, None)


@pytest.mark.parametrize("field,value", [
    ("score", 2), ("score", -1), ("group_score", 2), ("renorm", 2), ("groups", 0), ("groups", 3), ("groups", 128),
    ("kept_groups", 0), ("kept_groups", 5), ("kept_groups", 1), ("scale", float("nan")), ("scale", float("inf"))])
def test_bad_routers_are_refused(lib, field, value):  # noqa: F811
    # 128 experts in 4 groups of 32, 2 kept; k = 16
    s = shape_for(T=64, D=128, I=64, E=32, k=10)
    r = router_for(groups=4, kept_groups=2)
    setattr(r, field, value)
    assert call(lib, s, r) == -1
    assert call_backward(lib, s, r) == -1


def test_missing_arguments_are_refused(lib):  # noqa: F811
    s, r = shape_for(T=64, D=128, I=64, E=32, k=4), router_for()
    assert call(lib, s, None) == -1
    assert call_backward(lib, s, None) == -1
    for n in ("logits", "idx", "gate"):
        assert call(lib, s, r, **{n: None}) == -1, n
    assert call(lib, s, r, x=FAKE) == -1  # x without router weights
    for n in ("logits", "idx", "dgate", "out"):
        assert call_backward(lib, s, r, **{n: None}) == -1, n
    assert lib.moe_route_scored(ctypes.byref(s), ctypes.byref(r), None, None, None, FAKE, FAKE, FAKE, FAKE, 0,
                                None) == -3
    empty = shape_for(T=0, D=128, I=64, E=32, k=4)
    assert call(lib, empty, r) == 0 and call_backward(lib, empty, r) == 0  # nothing to do: no launch


def test_routing_without_tokens_still_checks_its_weights(lib):  # noqa: F811
    s, r = shape_for(T=0, D=128, I=64, E=32, k=4), router_for()
    n = ws_bytes(lib, s)[1]
    assert call(lib, s, r, logits=None, idx=None, gate=None) == 0
    assert call(lib, s, r, x=FAKE) == -1 and call(lib, s, None) == -1  # x without router weights, no router
    assert lib.moe_route(ctypes.byref(s), None, None, None, None, None, FAKE, n, None) == 0
    assert lib.moe_route(ctypes.byref(s), FAKE, None, FAKE, FAKE, FAKE, FAKE, n, None) == -1


def test_backward_scored_is_refused_like_backward(lib):  # noqa: F811
    s, r = shape_for(T=64, D=128, I=64, E=32, k=4), router_for()
    n = ctypes.c_size_t(0)
    assert lib.moe_backward_workspace_bytes(ctypes.byref(s), ctypes.byref(n)) == 0
    bw = _lib.MoeBwdWeights(*[4096] * len(_lib.MoeBwdWeights._fields_))
    g = _lib.MoeGrads(*[4096] * len(_lib.MoeGrads._fields_))

    def run(s, r, logits, ws):
        return lib.moe_backward_scored(ctypes.byref(s), r and ctypes.byref(r), ctypes.byref(bw), FAKE, logits, FAKE,
                                       FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(g), FAKE, FAKE, ws, None)
    assert run(s, None, FAKE, n.value) == -1
    assert run(s, r, None, n.value) == -1
    assert run(s, r, FAKE, n.value - 1) == -3
    assert run(shape_for(T=64, D=128, I=128, E=32, k=4, precision="mxfp8"), r, FAKE, n.value) == -2


def test_router_for_refuses_unknown_names():
    with pytest.raises(ValueError):
        router_for(score="relu")
    with pytest.raises(ValueError):
        router_for(group_score="mean")
