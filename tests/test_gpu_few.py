"""GPU parity of moe_few (the whole layer for a few tokens in one launch).

The reference is the layer in fp64 (torch on the device), with the choice taken
by the fp64 oracle from the GPU's own logits.  Bounds, with u = 2^-24:

* logits: fp32 sums of D exact products, in any order: D u sum |x| |w|.
* gates: fp64 from scores good to 1e-13, rounded once: u |g|, and 1e-12 for
  what renormalisation leaves.
* out32, bf16: h is kept to 2^-16 of its value (two bf16 terms, the second
  rounded: 2^-8 of 2^-8) and the sums before and after it to some sqrt(K) u of
  their terms' size, below that for K up to 7168 (85 * 2^-24 = 2^-17.6).  The errors
  of I values of h add at random in an output: 2^-16 of the RMS, and its largest of
  T D values (below 2^20) within 5.5 of that: 2^-13.5.  The bound is 2^-13 RMS.
* out32, MXFP8: values of x are quantised alike on both sides.  A value of h
  whose fp32 and fp64 forms (2^-18 apart) lie on two sides of a rounding
  border moves by a step, at most 2^-3 of it, and there are 2^-14 of them: one in
  most outputs' sums of I at the most, which moves by 2^-3 / sqrt(I) of its RMS,
  weighted by a gate: 5e-3 at I = 640 and 1.1e-2 at 128.  A block whose largest value
  lies at a power of two moves its 32 values so: 32^(1/2) as much, one block in 2^17.
  The bound is 2^-3 sqrt(32 / I) RMS.
* out is RNE(out32), bit for bit.
"""

import numpy as np
import pytest
import torch

from mixture_experts_layer_counts_amd import (MoELayer, pack_mxfp8_scales, quantize_mxfp8, router_for, shape_for,
                                              tile_bf16, tile_mxfp8)
from oracle import scored
from tests._gpu import need_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def mx_values(q, s):
    v = q.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
    return (v * torch.exp2(s.double() - 127).unsqueeze(-1)).flatten(-2)


def mx_round(v):
    """The values fp64 rows are stored as in MXFP8."""
    b = v.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(dim=-1, keepdim=True))
    X = torch.where(m > 0, e.double() - 9, -127.0).clamp(-127, 127)
    w = (b * torch.exp2(-X)).clamp(-448, 448)
    step = torch.exp2((torch.frexp(w)[1].double() - 4).clamp(min=-9))
    return (torch.round(w / step) * step * torch.exp2(X)).flatten(-2)


class Case:
    def __init__(self, dev, T, D, I, E, k, Is=None, prec="bf16", sprec="bf16", tiled=False, seed=0, x=None):
        Is = I if Is is None else Is
        g = torch.Generator(device=dev).manual_seed(seed)

        def rand(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device=dev) * std).to(torch.bfloat16)
        self.dev, self.T, self.D, self.I, self.E, self.k, self.Is = dev, T, D, I, E, k, Is
        self.x = rand(T, D) if x is None else x
        self.w_router = rand(E, D, std=D ** -0.5)
        self.weights, self.value = {}, {}
        for n, N, K in (("gate", I, D), ("up", I, D), ("down", D, I)):
            w = rand(E, N, K, std=K ** -0.5)
            if prec == "bf16":
                self.value[n] = w
                self.weights["w_" + n] = tile_bf16(w) if tiled else w
            else:
                q, s = quantize_mxfp8(w)
                self.value[n] = (q, s)
                self.weights["q_" + n] = tile_mxfp8(q) if tiled else q
                self.weights["s_" + n] = pack_mxfp8_scales(s)
        for n, N, K in (("gate", Is, D), ("up", Is, D), ("down", D, Is)):
            w = rand(N, K, std=K ** -0.5)
            if sprec == "bf16":
                self.value["s" + n] = w
                self.weights["ws_" + n] = w
            else:
                q, s = quantize_mxfp8(w)
                self.value["s" + n] = (q, s)
                self.weights["qs_" + n], self.weights["ss_" + n] = q, pack_mxfp8_scales(s.unsqueeze(0))[0]
        self.prec, self.sprec = prec, sprec
        self.layer = MoELayer(shape_for(T, D, I, E, k, I_shared=Is, precision=prec, shared_precision=sprec,
                                        weights_tiled=tiled), device=dev)

    def _ffn(self, x, pre, e, prec):
        def mat(n):
            v = self.value[pre + n]
            if prec == "bf16":
                return (v if e is None else v[e]).double()
            return mx_values(v[0], v[1]) if e is None else mx_values(v[0][e], v[1][e])
        q = mx_round if prec == "mxfp8" else (lambda v: v)
        a, u = q(x) @ mat("gate").T, q(x) @ mat("up").T
        return q(a / (1 + torch.exp(-a)) * u) @ mat("down").T

    def want(self, idx, gate):
        x = self.x.double()
        out = self._ffn(x, "s", None, self.sprec)
        for e in torch.unique(idx).tolist():
            t, s = torch.nonzero(idx == e, as_tuple=True)
            out[t] += gate[t, s].double()[:, None] * self._ffn(x[t], "", e, self.prec)
        return out

    def check(self, r, bias=None, from_x=True, **router):
        lg = r["logits"].cpu().numpy()
        if from_x:
            x, w = self.x.double(), self.w_router.double()
            err = (r["logits"].double() - x @ w.T).abs()
            assert bool((err <= self.D * U * (x.abs() @ w.abs().T)).all())
        kind = router.get("score", "softmax")
        s = scored.scores(lg, kind)
        b = None if bias is None else bias.cpu().numpy()
        idx = scored.choose(s, b, self.k, router.get("groups", 1), router.get("kept_groups", 1),
                            router.get("group_score", "top2"))
        assert np.array_equal(r["idx"].cpu().numpy(), idx)
        gate = scored.gates(s, idx, router.get("renorm", True), router.get("scale", 1.0))
        got = r["gate"].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - gate) <= U * np.abs(gate) + 1e-12 * router.get("scale", 1.0))
        want = self.want(r["idx"], r["gate"])
        err = float((r["out32"].double() - want).abs().max() / want.square().mean().sqrt())
        tol = 2.0 ** -13
        if "mxfp8" in (self.prec, self.sprec):
            tol = 2.0 ** -3 * (32 / min(self.I if self.prec == "mxfp8" else 1 << 20,
                                        self.Is if self.sprec == "mxfp8" else 1 << 20)) ** 0.5
        say("  max|err|/RMS =", err, "bound", tol)
        assert err <= tol
        assert torch.equal(r["out"], r["out32"].to(torch.bfloat16))
        assert self.layer.device_error() == 0


SIG = dict(score="sigmoid", groups=8, kept_groups=4, scale=2.5)
CASES = [  # T, D, I, E, k, Is, precision, shared precision, tiled, router
    (1, 64, 64, 1, 1, 64, "bf16", "bf16", False, None),
    (1, 128, 64, 8, 2, 64, "bf16", "bf16", False, None),
    (1, 2048, 768, 128, 8, 768, "bf16", "bf16", False, None),
    (2, 192, 320, 17, 3, 448, "bf16", "bf16", True, dict(score="sigmoid")),
    (3, 1472, 320, 100, 6, 704, "bf16", "bf16", False, dict(score="softmax", renorm=False)),
    (8, 512, 128, 256, 8, 64, "bf16", "bf16", True, SIG),
    (15, 256, 192, 40, 16, 128, "bf16", "bf16", False, dict(groups=4, kept_groups=2, group_score="max")),
    (16, 128, 64, 4, 4, 64, "bf16", "bf16", False, None),      # every token at every expert: full blocks
    (17, 128, 64, 3, 3, 64, "bf16", "bf16", True, None),       # one token past a block
    (33, 192, 128, 300, 5, 192, "bf16", "bf16", False, None),
    (64, 256, 64, 2, 1, 64, "bf16", "bf16", False, None),      # long lists
    (64, 128, 64, 1024, 16, 64, "bf16", "bf16", False, dict(score="sigmoid", groups=64, kept_groups=9)),
    (64, 2048, 768, 128, 8, 768, "bf16", "bf16", True, None),
    (1, 128, 128, 4, 2, 64, "mxfp8", "bf16", False, None),
    (5, 384, 256, 20, 4, 128, "mxfp8", "mxfp8", True, SIG | dict(groups=4, kept_groups=3)),
    (9, 640, 128, 12, 3, 256, "bf16", "mxfp8", False, None),
    (48, 512, 640, 16, 6, 192, "mxfp8", "bf16", True, None),
    (64, 256, 128, 6, 5, 384, "mxfp8", "mxfp8", False, None),
]


@pytest.mark.parametrize("T,D,I,E,k,Is,prec,sprec,tiled,router", CASES)
def test_layer(T, D, I, E, k, Is, prec, sprec, tiled, router):
    dev = need_gpu()
    say("few", T, D, I, E, k, Is, prec, sprec, tiled, router)
    c = Case(dev, T, D, I, E, k, Is, prec, sprec, tiled, seed=T + D)
    bias = None
    if router and router.get("groups", 1) > 1:
        bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1)).to(dev)
    r = c.layer.few(c.x, c.w_router, c.weights, router=router_for(**router) if router else None, bias=bias)
    c.check(r, bias, **(dict(score="sigmoid") | router if router else dict(score="softmax")))
    # again, and from the logits: the same bits, on a workspace that the last call left
    again = c.layer.few(c.x, c.w_router, c.weights, router=router_for(**router) if router else None, bias=bias)
    given = c.layer.few(c.x, None, c.weights, logits=r["logits"], router=router_for(**router) if router else None,
                        bias=bias)
    for n in ("logits", "idx", "gate", "out", "out32"):
        assert torch.equal(r[n], again[n]) and torch.equal(r[n], given[n]), n
    assert c.layer.few(c.x, c.w_router, c.weights, out32=False)["out32"] is None


def test_router_matches_the_standalone_one():
    """The same choice and the same gates, bit for bit, as moe_route_scored from the same logits."""
    dev = need_gpu()
    for E, k, kw in ((256, 8, SIG), (300, 5, dict(score="softmax", renorm=False)), (1000, 16, dict(groups=8, kept_groups=3)),
                     (7, 2, dict(score="softmax"))):
        c = Case(dev, 33, 64, 64, E, k, seed=E)
        bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(2)).to(dev)
        r = c.layer.few(c.x, c.w_router, c.weights, router=router_for(**kw), bias=bias)
        _, idx, gate = c.layer.route(None, None, r["logits"], router=router_for(**kw), bias=bias)
        assert torch.equal(idx, r["idx"]) and torch.equal(gate, r["gate"])


def test_odd_logits():
    """Given logits with ties, infinities, NaN and the type's lowest value: the choice and gates of moe_route_scored."""
    dev = need_gpu()
    low = torch.finfo(torch.float32).min
    for E, k, kw in ((40, 6, dict(score="sigmoid", groups=4, kept_groups=2)), (300, 16, dict(score="softmax")),
                     (700, 3, dict(score="softmax", renorm=False)), (64, 8, dict(groups=64, kept_groups=8, group_score="max"))):
        c = Case(dev, 12, 64, 64, E, k, seed=E)
        lg = torch.randn((12, E), generator=torch.Generator().manual_seed(E))
        lg[1] = lg[1].round()
        lg[2, ::3] = -float("inf")
        lg[3, 1::2] = float("nan")
        lg[4, 5:] = low
        lg[5] = -float("inf")
        lg[6] = 0.0
        lg[7, 7] = float("inf")
        lg = lg.to(dev)
        bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(2)).to(dev)
        for b in (None, bias):
            r = c.layer.few(c.x, None, c.weights, logits=lg, router=router_for(**kw), bias=b)
            assert c.layer.device_error() == 0x4  # MOE_DEVERR_NONFINITE
            _, idx, gate = c.layer.route(None, None, lg, router=router_for(**kw), bias=b)
            assert torch.equal(idx, r["idx"]) and torch.equal(gate, r["gate"])


def test_two_at_once():
    """Calls of two layers on two streams, and a captured one replayed beside eager calls of its own layer."""
    dev = need_gpu()
    a, b = Case(dev, 5, 1472, 320, 50, 6, 704, seed=1), Case(dev, 40, 512, 256, 30, 4, seed=2, tiled=True)
    want = [c.layer.few(c.x, c.w_router, c.weights) for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.layer.few(c.x, c.w_router, c.weights))
    torch.cuda.synchronize()
    for i in (0, 1):
        for r in got[i]:
            assert all(torch.equal(r[n], want[i][n]) for n in r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = a.layer.few(a.x, a.w_router, a.weights)
    for i in range(4):
        a.x.mul_(-1.5)
        graph.replay()
        w = a.layer.few(a.x, a.w_router, a.weights)
        torch.cuda.synchronize()
        assert all(torch.equal(r[n], w[n]) for n in r)
    assert a.layer.device_error() == 0 and b.layer.device_error() == 0


def test_tokens_do_not_meet():
    """A token's results are the same bits whatever the call's other tokens are, an infinity among them too."""
    dev = need_gpu()
    c = Case(dev, 20, 256, 128, 16, 4, seed=4)
    r = c.layer.few(c.x, c.w_router, c.weights)
    one = MoELayer(shape_for(1, 256, 128, 16, 4), device=dev)
    for t in (0, 7, 19):
        s = one.few(c.x[t:t + 1].contiguous(), c.w_router, c.weights)
        assert all(torch.equal(r[n][t:t + 1], s[n]) for n in r)
    c.x[3, 100] = float("inf")
    q = c.layer.few(c.x, c.w_router, c.weights)
    rest = [t for t in range(20) if t != 3]
    assert all(torch.equal(r[n][rest], q[n][rest]) for n in r)
    assert not torch.isfinite(q["out32"][3]).any()
    z = MoELayer(shape_for(0, 256, 128, 16, 4), device=dev).few(c.x[:0], c.w_router, c.weights)
    assert z["out"].shape == (0, 256)


def test_refusals():
    dev = need_gpu()
    c = Case(dev, 4, 128, 64, 8, 2)
    with pytest.raises(ValueError):
        c.layer.few(c.x[:3], c.w_router, c.weights)
    with pytest.raises(ValueError):
        c.layer.few(c.x, c.w_router, c.weights, bias=torch.zeros(8, device=dev))
    with pytest.raises(ValueError):
        c.layer.few(c.x.float(), c.w_router, c.weights)
    big = MoELayer(shape_for(65, 128, 64, 8, 2), device=dev)
    x = torch.zeros((65, 128), dtype=torch.bfloat16, device=dev)
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        big.few(x, c.w_router, c.weights)
    shifted = torch.zeros(4 * 128 + 1, dtype=torch.bfloat16, device=dev)[1:].view(4, 128)  # not 16-byte aligned
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        c.layer.few(shifted, c.w_router, c.weights)
