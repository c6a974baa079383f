"""GPU parity of moe_route_scored and moe_route_backward with the fp64 oracle.

The choice must equal the oracle's exactly.  Both sides form scores in fp64
(the kernel to 2^-42 for the choice); the seeded draws hold no two choosing
values closer than that.  Gates and gradients are computed in fp64 from scores
good to 1e-13 and rounded once, so the bound is half an fp32 step of the
value, 2^-24 |v|, plus what the cancellation in dg_s - mean leaves.  The terms
that cancel there are s/W scale dg <= scale max|dg| (s <= W; without
renormalisation s <= 1), and each is carried to about 1e-13: 1e-12 scale
max|dg|.  (With one expert a token, dg - mean is zero but for that, and the
gradient has no larger entry to measure it by.)
"""

import numpy as np
import pytest
import torch

import synth
from mixture_experts_layer_counts_amd import MoEBackward, MoELayer, prepare_backward, router_for, shape_for
from oracle import bf16, scored
from tests._gpu import host_weights, layer, need_gpu, rel_err, say, to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def close(got, want, dg=None, scale=1.0):
    """dg: the gradient of the gates, when `want` is the logits' gradient for it."""
    want = np.asarray(want, dtype=np.float64)
    terms = np.abs(want if dg is None else scale * np.asarray(dg)).max(axis=-1, keepdims=True)
    tol = U * np.abs(want) + 1e-12 * terms + 1e-44
    return np.all(np.abs(np.asarray(got, dtype=np.float64) - want) <= tol)


def run(dev, logits, k, bias=None, **kw):
    T, E = logits.shape
    m = MoELayer(shape_for(T, 128, 64, E, k), device=dev)
    r = router_for(**kw)
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).to(dev)
    lg = torch.from_numpy(logits.astype(np.float32)).to(dev)
    _, idx, gate = m.route(None, None, lg, router=r, bias=b)
    return m, r, lg, idx, gate


CASES = [  # T, E, k, bias, router
    (1, 256, 8, True, dict(score="sigmoid", groups=8, kept_groups=4, scale=2.5)),
    (300, 256, 8, True, dict(score="sigmoid", groups=8, kept_groups=4, scale=2.5)),
    (301, 256, 8, False, dict(score="softmax")),
    (67, 384, 6, False, dict(score="softmax", groups=12, kept_groups=5, group_score="max", renorm=False)),
    (33, 1024, 16, True, dict(score="sigmoid", groups=64, kept_groups=9, renorm=False)),
    (19, 1000, 16, True, dict(score="softmax", groups=8, kept_groups=3, renorm=False, scale=16.0)),
    (5, 1, 1, False, dict(score="sigmoid")),
    (9, 3, 3, True, dict(score="softmax", groups=3, kept_groups=3)),
    (130, 7, 2, False, dict(score="sigmoid", renorm=False)),
    (65, 60, 5, True, dict(score="sigmoid", groups=20, kept_groups=2)),
    (40, 66, 4, True, dict(score="softmax", groups=33, kept_groups=2, group_score="max")),
    (77, 513, 9, False, dict(score="sigmoid", groups=27, kept_groups=13)),
    (50, 64, 8, True, dict(score="softmax", groups=64, kept_groups=8)),
    (128, 100, 12, False, dict(score="sigmoid", groups=2, kept_groups=1, group_score="max")),
    # enough tokens that several share a wave
    (2101, 256, 8, True, dict(score="sigmoid", groups=8, kept_groups=4, scale=2.5)),
    (2060, 100, 12, True, dict(score="softmax", groups=25, kept_groups=7)),
    (2049, 384, 6, False, dict(score="softmax", groups=12, kept_groups=5, group_score="max", renorm=False)),
    (2051, 500, 16, True, dict(score="sigmoid", groups=20, kept_groups=3)),
    (2050, 128, 9, False, dict(score="sigmoid", groups=4, kept_groups=1)),
    (2053, 201, 3, True, dict(score="softmax", renorm=False)),
    # every count of lanes and experts a lane with up to 8 and up to 16 choices
    (31, 500, 16, False, dict(score="softmax", groups=4, kept_groups=2, group_score="max")),
    (2055, 256, 11, False, dict(score="sigmoid", groups=16, kept_groups=5)),
    (1030, 120, 8, True, dict(score="sigmoid", groups=15, kept_groups=4)),
    (1031, 300, 10, False, dict(score="sigmoid", groups=3, kept_groups=1, group_score="max")),
    (1033, 512, 7, True, dict(score="softmax", groups=32, kept_groups=4)),
    (41, 640, 8, True, dict(score="sigmoid", groups=5, kept_groups=2)),
    # either side of where a wave takes a token
    (1024, 128, 4, True, dict(score="sigmoid", groups=8, kept_groups=2)),
    (1025, 128, 4, True, dict(score="sigmoid", groups=8, kept_groups=2)),
    (2048, 160, 4, False, dict(score="softmax", groups=10, kept_groups=3)),
    (1025, 260, 6, False, dict(score="softmax")),
]


@pytest.mark.parametrize("T,E,k,bias,kw", CASES, ids=[f"{c[0]}x{c[1]}k{c[2]}" for c in CASES])
def test_route_scored_parity(T, E, k, bias, kw):
    dev = need_gpu()
    say("route_scored", T, E, k, kw)
    rng = np.random.default_rng(T * 7 + E)
    logits = (2.0 * rng.standard_normal((T, E))).astype(np.float32)
    b = (0.2 * rng.standard_normal(E)).astype(np.float32) if bias else None
    m, r, lg, idx, gate = run(dev, logits, k, b, **kw)
    torch.cuda.synchronize()
    assert m.device_error() == 0
    kind, renorm, scale = kw["score"], kw.get("renorm", True), kw.get("scale", 1.0)
    s = scored.scores(logits, kind)
    want = scored.choose(s, b, k, kw.get("groups", 1), kw.get("kept_groups", 1), kw.get("group_score", "top2"))
    assert np.array_equal(idx.cpu().numpy(), want)
    assert close(gate.cpu().numpy(), scored.gates(s, want, renorm, scale))
    dg = rng.standard_normal((T, k)).astype(np.float32)
    dl = m.route_backward(lg, idx, torch.from_numpy(dg).to(dev), router=r)
    torch.cuda.synchronize()
    assert m.device_error() == 0
    got = dl.cpu().numpy()
    assert close(got, scored.backward(logits, want, dg, kind, renorm, scale), dg, scale)
    if kind == "sigmoid" or renorm:
        off = np.ones((T, E), dtype=bool)
        np.put_along_axis(off, want.astype(np.int64), False, axis=1)
        assert np.all(got[off] == 0)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_ties_go_to_the_lower_id(kind):
    dev = need_gpu()
    say("route_scored ties", kind)
    logits = np.zeros((6, 256), dtype=np.float32)
    logits[1, 200:] = 1.0
    logits[2] = np.repeat(np.arange(8)[::-1], 32)  # whole groups of equal logits
    logits[3] = -0.0
    logits[4, ::2] = 0.5
    logits[5] = -60.0  # every score tiny
    for kw in (dict(), dict(groups=8, kept_groups=3), dict(groups=8, kept_groups=3, group_score="max")):
        m, _, _, idx, gate = run(dev, logits, 8, score=kind, **kw)
        s = scored.scores(logits, kind)
        want = scored.choose(s, None, 8, kw.get("groups", 1), kw.get("kept_groups", 1), kw.get("group_score", "top2"))
        assert np.array_equal(idx.cpu().numpy(), want), kw
        assert close(gate.cpu().numpy(), scored.gates(s, want, True, 1.0))
        assert m.device_error() == 0


def test_negative_choosing_values():
    # a bias that takes every c below zero keeps the order and the tie rule
    dev = need_gpu()
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((40, 96)).astype(np.float32)
    logits[:8] = 0.25
    bias = np.full(96, -3.0, dtype=np.float32)
    bias[::3] = -2.5
    m, _, _, idx, _ = run(dev, logits, 7, bias, score="sigmoid", groups=6, kept_groups=2)
    want = scored.choose(scored.scores(logits, "sigmoid"), bias, 7, 6, 2)
    assert np.array_equal(idx.cpu().numpy(), want) and m.device_error() == 0


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_and_nonfinite_logits(kind, renorm):
    # -inf masks an expert (score 0); a row of nothing but masks has zero gates;
    # NaN counts as -inf; each sets the error bit
    dev = need_gpu()
    say("route_scored masked", kind, renorm)
    rng = np.random.default_rng(11)
    logits = rng.standard_normal((5, 32)).astype(np.float32)
    logits[0, 3:] = -np.inf
    logits[1, :] = -np.inf
    logits[2, ::2] = -np.inf
    logits[3, 5] = np.nan
    lowest = torch.finfo(torch.float32).min
    logits[4, 1:] = lowest  # the type's lowest value is a number: no flag of its own
    m, r, lg, idx, gate = run(dev, logits, 4, score=kind, renorm=renorm)
    assert m.device_error() == 0x4
    clean = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    s = scored.scores(clean, kind)
    want = scored.choose(s, None, 4)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert close(gate.cpu().numpy(), scored.gates(s, want, renorm, 1.0))
    if renorm:
        assert np.all(gate.cpu().numpy()[1] == 0)
    dg = rng.standard_normal((5, 4)).astype(np.float32)
    got = m.route_backward(lg, idx, torch.from_numpy(dg).to(dev), router=r).cpu().numpy()
    assert close(got, scored.backward(clean, want, dg, kind, renorm, 1.0), dg)
    # infinite logits and biases choose as they compare, and are flagged
    logits = rng.standard_normal((3, 32)).astype(np.float32)
    logits[1, 9] = np.inf
    bias = np.zeros(32, dtype=np.float32)
    bias[20], bias[2], bias[0] = np.inf, -np.inf, np.nan
    m, _, _, idx, gate = run(dev, logits, 2, bias, score=kind, renorm=renorm)
    assert m.device_error() == 0x4
    got = idx.cpu().numpy()
    assert np.all(got[:, 0] == 20) and got[1, 1] == 9 and not np.isin(got, (0, 2)).any()
    assert torch.isfinite(gate).all()


def test_route_backward_refuses_ids_out_of_range():
    dev = need_gpu()
    logits = np.random.default_rng(0).standard_normal((4, 16)).astype(np.float32)
    m, r, lg, idx, _ = run(dev, logits, 3, score="softmax", renorm=False)
    good = idx.cpu().numpy()
    dg = torch.ones((4, 3), device=dev)
    bad = idx.clone()
    bad[1, 2], bad[2, 0] = 16, -1
    got = m.route_backward(lg, bad, dg, router=r).cpu().numpy()
    assert m.device_error() & 0x1
    want = scored.backward(logits, good, np.ones((4, 3)), "softmax", False, 1.0)
    assert close(got[[0, 3]], want[[0, 3]], np.ones((2, 3)))
    drop = np.ones((4, 3))
    drop[1, 2] = drop[2, 0] = 0.0  # what a slot that adds nothing leaves
    assert close(got, scored.backward(logits, good, drop, "softmax", False, 1.0), np.ones((4, 3)))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_gradient_of_a_single_renormalised_gate_is_zero(kind):
    # the gate is `scale` whatever the logit
    dev = need_gpu()
    say("one expert a token", kind)
    for T, E in ((1, 6), (17, 36), (3000, 300)):
        rng = np.random.default_rng(E)
        m, r, lg, idx, gate = run(dev, rng.standard_normal((T, E)), 1, score=kind, scale=2.5)
        dg = torch.from_numpy(rng.standard_normal((T, 1)).astype(np.float32)).to(dev)
        assert torch.all(gate == 2.5)
        assert not m.route_backward(lg, idx, dg, router=r).any()


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_saturated_sigmoids(renorm):
    # 1 - s of a score next to 1 is what the gradient is made of: right relative to itself, out to the fp32 range
    dev = need_gpu()
    say("saturated sigmoids", renorm)
    rng = np.random.default_rng(8)
    for T, E, k in ((40, 64, 6), (2100, 256, 8)):
        logits = rng.uniform(20.0, 60.0, (T, E)).astype(np.float32)
        logits[1::3] *= -1.0
        logits[2::3, ::2] *= -1.0
        m, r, lg, idx, _ = run(dev, logits, k, score="sigmoid", renorm=renorm, scale=2.5)
        dg = rng.standard_normal((T, k)).astype(np.float32)
        got = m.route_backward(lg, idx, torch.from_numpy(dg).to(dev), router=r).cpu().numpy().astype(np.float64)
        ids = idx.cpu().numpy()
        want = scored.backward(logits, ids, dg, "sigmoid", renorm, 2.5)
        # half an fp32 step, and 1e-12 of the terms that cancel in dg_s - mean, each times scale s (1 - s) / W
        s = scored.scores(logits, "sigmoid")
        W = np.take_along_axis(s, ids.astype(np.int64), axis=1).sum(1, keepdims=True) if renorm else 1.0
        unit = 2.5 * s * scored.scores(-logits, "sigmoid") / W
        tol = U * np.abs(want) + 1e-12 * unit * np.abs(dg).max(1, keepdims=True)
        assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(40, 64, 5), (2100, 256, 8), (1100, 300, 12)])
def test_renormalised_gates_of_logits_far_below_the_others(kind, T, E, k):
    # a bias that chooses masked experts (finite masks, and the type's lowest value): the gates depend on the chosen
    # logits' differences alone, forward and backward
    dev = need_gpu()
    say("far below", kind, T, E, k)
    rng = np.random.default_rng(E)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    chosen = rng.permutation(E)[:k]
    bias = np.zeros(E, dtype=np.float32)
    bias[chosen] = 10.0 + np.arange(k)[::-1]  # in this order, whatever the scores
    depth = np.array([-1e4, -499.0, -501.0, -650.0, -699.0, -720.0, -3e5, 0.0])
    logits[:, chosen] += depth[np.arange(T) % 8][:, None].astype(np.float32)
    logits[::16, chosen] = torch.finfo(torch.float32).min
    logits[5::16, chosen[1:]] -= 5e3  # one of them far above the rest
    m, r, lg, idx, gate = run(dev, logits, k, bias, score=kind, scale=2.5)
    ids = idx.cpu().numpy()
    assert np.array_equal(ids, np.tile(chosen, (T, 1))) and m.device_error() == 0
    assert close(gate.cpu().numpy(), 2.5 * scored.ratios(logits, ids, kind))
    assert np.allclose(gate.double().sum(1).cpu().numpy(), 2.5, rtol=k * U, atol=0)
    dg = rng.standard_normal((T, k)).astype(np.float32)
    got = m.route_backward(lg, idx, torch.from_numpy(dg).to(dev), router=r).cpu().numpy()
    assert close(got, scored.backward(logits, ids, dg, kind, True, 2.5), dg, 2.5)


def test_routing_from_x_scores_the_same_logits():
    # the router projection with K ranges: the choice equals the oracle's of the logits that come back
    dev = need_gpu()
    w = synth.Workload("scored-x", T=513, D=1024, I=64, E=256, k=8, I_shared=64, seed=9)
    inp = to_dev(synth.make_inputs(w), dev)
    m = layer(w, dev)
    r = router_for(score="sigmoid", groups=8, kept_groups=4, scale=2.5)
    lg, idx, gate = m.route(inp["x"], inp["w_router"], router=r)
    plain, _, _ = m.route(inp["x"], inp["w_router"])
    assert torch.equal(lg, plain)
    s = scored.scores(lg.cpu().numpy(), "sigmoid")
    want = scored.choose(s, None, 8, 8, 4)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert close(gate.cpu().numpy(), scored.gates(s, want, True, 2.5))
    assert m.device_error() == 0


def test_softmax_router_agrees_with_moe_route():
    dev = need_gpu()
    logits = torch.randn((777, 128), generator=torch.Generator().manual_seed(1)).to(dev)
    m = MoELayer(shape_for(777, 128, 64, 128, 8), device=dev)
    _, i0, g0 = m.route(None, None, logits)
    _, i1, g1 = m.route(None, None, logits, router=router_for(score="softmax"))
    assert torch.equal(i0, i1)
    # moe_route's gates are fp32 arithmetic: 2 max|l_s - l_0| + k + 8 rounding units, logits within +-6
    assert torch.all((g0 - g1).abs() <= U * (2 * 12 + 8 + 8) * g1)


def test_unaligned_logits():
    # logits that start 4 bytes past an aligned address
    dev = need_gpu()
    T, E = 37, 64
    buf = torch.randn(T * E + 1, generator=torch.Generator().manual_seed(2)).to(dev)
    m = MoELayer(shape_for(T, 128, 64, E, 4), device=dev)
    r = router_for(score="sigmoid")
    view = buf[1:].view(T, E)
    a = m.route(None, None, view, router=r)
    b = m.route(None, None, view.clone(), router=r)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    dg = torch.ones((T, 4), device=dev)
    assert torch.equal(m.route_backward(view, a[1], dg, router=r), m.route_backward(view.clone(), a[1], dg, router=r))


def scored_layer(dev, w, kw, bias):
    """A forward with a scored router, and both backwards of its gates."""
    inp = synth.make_inputs(w)
    d = to_dev(inp, dev)
    m = layer(w, dev)
    r = router_for(**kw)
    res = m(d["x"], d["w_router"], d, logits=d["logits"], router=r, bias=bias)
    y = m.routed_rows().clone()
    bw = prepare_backward(m.shape, d, d["w_router"])
    back = MoEBackward(m.shape, device=dev)
    dout = torch.randn((w.T, w.D), generator=torch.Generator().manual_seed(w.seed + 5)).to(torch.bfloat16).to(dev)
    return inp, d, m, r, res, y, bw, back, dout


@pytest.mark.parametrize("kw", [dict(score="sigmoid", groups=4, kept_groups=2, scale=2.5),
                                dict(score="softmax", renorm=False, scale=1.5), dict(score="softmax")],
                         ids=["sigmoid", "softmax", "softmax-renorm"])
def test_layer_backward_with_a_scored_router(kw):
    """The whole layer under a scored router: the expert gradients are those of
    moe_backward on the same gates bit for bit, dW_r = r(dl)^T x with dl from the
    oracle, and dx differs from moe_backward's by the two routers' shares."""
    dev = need_gpu()
    w = synth.Workload("scored-layer", T=300, D=256, I=192, E=16, k=4, I_shared=128, seed=7, routing="gaussian")
    say("backward_scored", kw)
    bias = torch.linspace(-0.2, 0.2, w.E, device=dev)
    inp, d, m, r, res, y, bw, back, dout = scored_layer(dev, w, kw, bias)
    got = back(bw, d["x"], res["idx"], res["gate"], res, y, dout, router=r, logits=res["logits"])
    plain = back(bw, d["x"], res["idx"], res["gate"], res, y, dout)
    torch.cuda.synchronize()
    assert m.device_error() == 0 and back.device_error() == 0
    for n in ("dw_gate", "dw_up", "dw_down", "dws_gate", "dws_up", "dws_down"):
        assert torch.equal(got[n], plain[n]), n
    idx, g = res["idx"].cpu().numpy(), res["gate"].double().cpu().numpy()
    do = bf16.to_f64(synth.bits(dout.cpu()))
    dg = np.einsum("td,tsd->ts", do, y.double().cpu().numpy().reshape(w.T, w.k, w.D))
    lg = inp["logits"].numpy()
    dl = scored.backward(lg, idx, dg, kw["score"], kw.get("renorm", True), kw.get("scale", 1.0))
    x, wr = inp["x"].double().numpy(), inp["w_router"].double().numpy()

    def r16(v):
        return torch.from_numpy(v).to(torch.bfloat16).double().numpy()
    # 1e-2 RMS: the bound of the other fp32 gradients (dl is stored bf16 on both sides)
    assert rel_err(got["dw_router"].cpu().numpy(), r16(dl).T @ x) <= 1e-2
    own = np.zeros_like(dl)
    np.put_along_axis(own, idx.astype(np.int64), g * (dg - (g * dg).sum(1, keepdims=True)), axis=1)
    want = plain["dx"].double().cpu().numpy() + (r16(dl) - r16(own)) @ wr
    assert rel_err(got["dx"].cpu().numpy(), want) <= 1e-2
    again = back(bw, d["x"], res["idx"], res["gate"], res, y, dout, router=r, logits=res["logits"])
    for n in got:
        assert torch.equal(got[n], again[n]), n


def test_scored_routing_in_a_graph_and_on_another_stream():
    dev = need_gpu()
    T, E, k = 600, 256, 8
    say("route_scored graph")
    m = MoELayer(shape_for(T, 128, 64, E, k), device=dev)
    r = router_for(score="sigmoid", groups=8, kept_groups=4, scale=2.5)
    gen = torch.Generator().manual_seed(6)
    logits, dg = torch.randn((T, E), generator=gen).to(dev), torch.randn((T, k), generator=gen).to(dev)
    bias = 0.1 * torch.randn(E, generator=gen).to(dev)

    def step():
        _, idx, gate = m.route(None, None, logits, router=r, bias=bias)
        return idx, gate, m.route_backward(logits, idx, dg, router=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for rep in range(3):
        logits.copy_(torch.randn((T, E), generator=gen))
        want = [v.clone() for v in step()]
        for v in got:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep
