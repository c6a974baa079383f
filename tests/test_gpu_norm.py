"""GPU parity of moe_block_norm and moe_block_norm_backward with their formulas in
fp64, differentiated by torch, and of the dropout mask with Philox's published
answers.

Bounds, with u = 2^-24 (an fp32 rounding) and e the half step of an output's type
(2^-9 of its value in bf16, u in fp32: RNE is off by at most half a step):

* rows (z, h, dx, dy): a chain of some twenty fp32 operations on terms no
  larger than ``terms`` (the sum of the absolute terms that make up the value),
  and row sums of D squares or products, whose relative error is at most
  (D / 8 + 16) u (8 or 16 values a thread in a chain, then a tree over the threads:
  16 + 12 additions at most): 64 u in all, times the terms, plus e of the value.
* column sums: T terms added in chains of the run's rows (at most
  ceil(T 2^-10) + 8) and then over at most 1024 runs in 16 chains: the sum of
  their absolute values times (T / 64 + 160) u.
"""

import numpy as np
import pytest
import torch

from mixture_experts_layer_counts_amd import block_norm, block_norm_backward
from tests._gpu import need_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def philox(c, k):
    c, k = list(c), list(k)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def mask(T, D, p, seed, offset):
    """The kept elements, in Python's integers."""
    out = np.zeros((T, D), dtype=bool)
    limit = round(p * 2 ** 32)
    for t in range(T):
        for q in range((D + 3) // 4):
            w = philox((q, t, offset & 0xFFFFFFFF, offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
            for i in range(4):
                if 4 * q + i < D:
                    out[t, 4 * q + i] = w[i] >= limit
    return torch.from_numpy(out)


def test_philox_known_answers():
    # the generator's published test vectors (random123's kat_vectors, philox4x32 10)
    assert philox((0, 0, 0, 0), (0, 0)) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    f = 0xFFFFFFFF
    assert philox((f, f, f, f), (f, f)) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert philox((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0)) == [
        0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


class Case:
    def __init__(self, dev, T, D, xt, yt, wt, ht, post, G, pre, p, scale=1.0, offset=0.0, has_y=True, seed=0):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape, dt, add=0.0):
            return (torch.randn(shape, generator=g) + add).to(dt).to(dev)
        ch = torch.exp(0.5 * torch.randn(D, generator=g))
        self.x = (torch.randn((T, D), generator=g) * ch).to(xt).to(dev)
        self.y = (torch.randn((T, D), generator=g) * ch).to(yt).to(dev) if has_y else None
        self.dz = rand(T, D, dt=xt)
        self.dh = rand(T, D, dt=ht) if pre else None
        self.seed, self.off = 0x123456789ABCDEF0 + seed, 0x0FEDCBA987654321
        rng = torch.tensor([self.seed, self.off], dtype=torch.int64, device=dev) if p else None
        self.kw = dict(post_weight=rand(D, dt=wt, add=1.0 - offset) if post else None,
                       gate=rand(G, D, dt=wt) if G else None,
                       pre_weight=rand(D, dt=wt, add=1.0 - offset) if pre else None,
                       scale=scale, eps=EPS, weight_offset=offset, dropout=p, rng=rng)
        self.T, self.D, self.p = T, D, p
        self.keep = mask(T, D, p, self.seed, self.off).to(dev) if p else None

    def leaves(self):
        names = {"x": self.x, "y": self.y, "post": self.kw["post_weight"], "gate": self.kw["gate"],
                 "pre": self.kw["pre_weight"]}
        return {n: None if v is None else v.double().requires_grad_() for n, v in names.items()}

    def term(self, v):
        """What is added to x, in fp64."""
        off = self.kw["weight_offset"]
        n = v["y"]
        if v["post"] is not None:
            n = n * torch.rsqrt(n.square().mean(1, keepdim=True) + EPS) * (v["post"] + off)
        if v["gate"] is not None:
            n = n * v["gate"].repeat_interleave(self.T // v["gate"].shape[0], 0)
        n = n * (self.kw["scale"] / (1 - self.p))
        return n if self.keep is None else torch.where(self.keep, n, 0.0)

    def out(self, v, z):
        if v["pre"] is None:
            return None
        return z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * (v["pre"] + self.kw["weight_offset"])


def half(dt):
    return torch.finfo(dt).eps / 2


def near(name, got, want, terms, n=64.0):
    # (2^-140: what a product below fp32's normal range may lose)
    tol = half(got.dtype) * want.abs() + n * U * terms + 2.0 ** -140
    err = (got.double() - want).abs()
    worst = float((err / tol).max()) if err.numel() else 0.0
    say("  ", name, "worst error / bound", worst)
    assert worst <= 1.0, name


def check_forward(c):
    z, h = block_norm(c.x, c.y, **c.kw)
    with torch.no_grad():
        v = c.leaves()
        add = c.term(v) if c.y is not None else torch.zeros_like(c.x, dtype=torch.float64)
        want = c.x.double() + add
        if c.y is None:
            assert z is c.x
        else:
            near("z", z, want, c.x.double().abs() + add.abs())
        if h is None:
            assert c.kw["pre_weight"] is None
        else:
            r = torch.rsqrt(want.square().mean(1, keepdim=True) + EPS)
            near("h", h, c.out(v, want), (c.x.double().abs() + add.abs()) * r * (v["pre"] + c.kw["weight_offset"]).abs())
    z2, h2 = block_norm(c.x, c.y, **c.kw)
    assert torch.equal(z, z2) and (h is None or torch.equal(h, h2))
    return z, h


def check_backward(c, with_dz=True):
    z = c.x  # any stream will do for z: the gradient is a function of it
    g = block_norm_backward(z, c.y, c.dz if with_dz else None, c.dh, **c.kw)
    v = c.leaves()
    if c.y is not None:
        n = c.term(v)
        zz = v["x"] + (n - n.detach())
    else:
        zz = v["x"]
    total = (zz * c.dz.double()).sum() if with_dz else zz.sum() * 0.0
    h = c.out(v, zz)
    if h is not None:
        total = total + (h * c.dh.double()).sum()
    total.backward()
    off = c.kw["weight_offset"]
    with torch.no_grad():
        rms = lambda t: t.square().mean(1, keepdim=True).sqrt()  # noqa: E731
        zd = z.double()
        parts = c.dz.double().abs() if with_dz else torch.zeros_like(zd)
        cols = {}
        if h is not None:
            r = torch.rsqrt(zd.square().mean(1, keepdim=True) + EPS)
            a = c.dh.double() * (v["pre"] + off)
            # mean(a z) r is at most the RMS of a, times z r
            parts = parts + r * (a.abs() + (zd * r).abs() * rms(a))
            cols["dpre_weight"] = (v["pre"].grad, (c.dh.double() * zd * r).abs().sum(0))
        near("dx", g["dx"], v["x"].grad, parts)
        if c.y is not None:
            f = c.kw["scale"] / (1 - c.p) * (1.0 if c.keep is None else c.keep.double())
            dn = parts * abs(f) if isinstance(f, float) else parts * f.abs()
            y = c.y.double()
            ry = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) if v["post"] is not None else torch.ones_like(y[:, :1])
            w = (v["post"] + off).abs() if v["post"] is not None else 1.0
            gv = v["gate"].repeat_interleave(c.T // v["gate"].shape[0], 0).abs() if v["gate"] is not None else 1.0
            b = dn * gv * w
            near("dy", g["dy"], v["y"].grad, ry * (b + (y * ry).abs() * rms(b)) if v["post"] is not None else b, n=128.0)
            if v["post"] is not None:
                cols["dpost_weight"] = (v["post"].grad, (dn * gv * (y * ry).abs()).sum(0))
            if v["gate"] is not None:
                G = v["gate"].shape[0]
                cols["dgate"] = (v["gate"].grad, (dn * (y * ry).abs() * w).view(G, c.T // G, c.D).sum(1))
        for n, (want, terms) in cols.items():
            near(n, g[n], want, terms, n=c.T / 64 + 160.0)
    for n, present in (("dy", c.y), ("dpost_weight", c.kw["post_weight"]), ("dgate", c.kw["gate"]),
                       ("dpre_weight", c.kw["pre_weight"])):
        assert (g[n] is None) == (present is None)
    again = block_norm_backward(z, c.y, c.dz if with_dz else None, c.dh, **c.kw)
    for n in g:
        assert g[n] is None or torch.equal(g[n], again[n]), n
    return g


CASES = [  # T, D, x, y, w, dh, post, G, pre, dropout, scale, offset
    (1, 8, BF, BF, BF, BF, True, 0, True, 0.0, 1.0, 0.0),
    (1, 7168, BF, BF, BF, F32, True, 1, True, 0.0, 1.0, 0.0),
    (3, 9, F32, BF, F32, BF, True, 3, True, 0.25, 0.5, 1.0),
    (5, 15, BF, F32, BF, F32, False, 1, True, 0.5, 1.0, 0.0),
    (7, 64, BF, BF, F32, BF, True, 7, False, 0.1, 1.0, 0.0),
    (16, 100, F32, F32, F32, F32, False, 0, True, 0.0, 0.22, 0.0),
    (33, 513, BF, BF, BF, BF, True, 1, True, 0.1, 1.0, 1.0),
    (64, 1001, F32, F32, F32, F32, True, 8, True, 0.1, 0.5, 0.0),
    (257, 1024, BF, BF, BF, F32, True, 1, True, 0.0, 1.0, 0.0),
    (300, 72, BF, BF, BF, BF, True, 100, True, 0.0, 1.0, 0.0),
    (1030, 40, F32, BF, BF, F32, True, 2, True, 0.0, 1.0, 0.0),
    (3000, 24, BF, F32, F32, BF, True, 3000, True, 0.0, 1.0, 0.0),
    (20, 8192, BF, BF, BF, BF, True, 1, True, 0.0, 1.0, 0.0),
    (9, 8193, F32, F32, F32, F32, True, 3, True, 0.0, 1.0, 0.0),
    (6, 16384, BF, F32, BF, F32, True, 1, True, 0.1, 1.0, 0.0),
    (11, 10007, BF, BF, F32, BF, False, 11, False, 0.0, 1.0, 0.0),
    (70, 2048, BF, BF, BF, BF, False, 0, False, 0.3, 1.0, 0.0),
]


@pytest.mark.parametrize("T,D,xt,yt,wt,ht,post,G,pre,p,scale,offset", CASES)
def test_against_formulas(T, D, xt, yt, wt, ht, post, G, pre, p, scale, offset):
    dev = need_gpu()
    say("norm", T, D, xt, yt, wt, ht, post, G, pre, p)
    c = Case(dev, T, D, xt, yt, wt, ht, post, G, pre, p, scale, offset, seed=T + D)
    check_forward(c)
    check_backward(c)
    if pre:
        check_backward(c, with_dz=False)


@pytest.mark.parametrize("T,D,xt,wt", [(1, 2048, BF, BF), (130, 999, F32, F32), (19, 9000, BF, F32)])
def test_without_y(T, D, xt, wt):
    dev = need_gpu()
    c = Case(dev, T, D, xt, BF, wt, F32, False, 0, True, 0.0, has_y=False, seed=3)
    check_forward(c)
    check_backward(c)


def test_long_runs():
    """More rows than one round of teams, groups across the ends of runs."""
    dev = need_gpu()
    for T, G in ((40000, 4), (40001, 1), (16384, 64)):
        c = Case(dev, T, 24, BF, BF, BF, F32, True, G, True, 0.0, seed=T)
        check_forward(c)
        check_backward(c)


def test_differences():
    """The gradients against central differences of the kernel's own fp32 forward, in the directions of
    random vectors.  With a step s the difference is off by s^2 / 6 of the third derivative and by the forward's
    rounding over s: at s = 2^-6 both are below 2e-3 of the products' sizes here."""
    dev = need_gpu()
    c = Case(dev, 12, 96, F32, F32, F32, F32, True, 3, True, 0.2, scale=0.7, seed=5)
    z, h = block_norm(c.x, c.y, **c.kw)
    dz, dh = c.dz, c.dh
    g = block_norm_backward(z, c.y, dz, dh, **c.kw)
    gen = torch.Generator().manual_seed(9)

    def loss(x, y, kw):
        # z alone: h is rounded to bf16, too coarse for differences; h enters through its own norm of z
        zz, _ = block_norm(x, y, **{**kw, "pre_weight": None})
        r = torch.rsqrt(zz.double().square().mean(1, keepdim=True) + EPS)
        hh = zz.double() * r * kw["pre_weight"].double()
        return float((zz.double() * dz.double()).sum() + (hh * dh.double()).sum())
    for name, grad in (("x", "dx"), ("y", "dy"), ("post_weight", "dpost_weight"), ("gate", "dgate"),
                       ("pre_weight", "dpre_weight")):
        base = {"x": c.x, "y": c.y}.get(name, c.kw.get(name))
        v = torch.randn(base.shape, generator=gen).to(dev)
        s = 2.0 ** -6
        ends = []
        for sign in (1.0, -1.0):
            moved = base + sign * s * v
            x, y, kw = c.x, c.y, dict(c.kw)
            if name == "x":
                x = moved
            elif name == "y":
                y = moved
            else:
                kw[name] = moved
            ends.append(loss(x, y, kw))
        diff = (ends[0] - ends[1]) / (2 * s)
        want = float((g[grad].double() * v.double()).sum())
        size = float((g[grad].double().square().sum() * v.double().square().sum()).sqrt())
        say("  ", name, diff, want, abs(diff - want) / size)
        assert abs(diff - want) <= 2e-3 * size, name


def test_masked_values():
    """A dropped infinity or NaN adds nothing; kept ones and those of the stream go through."""
    dev = need_gpu()
    c = Case(dev, 8, 64, BF, BF, BF, BF, False, 1, False, 0.5, seed=1)
    dropped = ~c.keep
    y = c.y.clone()
    y[dropped] = float("inf")
    y[0, dropped[0]] = float("nan")
    z, _ = block_norm(c.x, y, **c.kw)
    z0, _ = block_norm(c.x, c.y, **c.kw)
    assert torch.equal(z, z0)
    g = block_norm_backward(z, y, c.dz, None, **c.kw)
    g0 = block_norm_backward(z, c.y, c.dz, None, **c.kw)
    for n in ("dx", "dy", "dgate"):
        assert torch.equal(g[n], g0[n]), n


def test_no_rows():
    dev = need_gpu()
    x = torch.zeros((0, 64), dtype=BF, device=dev)
    w = torch.ones(64, dtype=BF, device=dev)
    z, h = block_norm(x, x.clone(), post_weight=w, pre_weight=w)
    assert z.shape == (0, 64) and h.shape == (0, 64)
    g = block_norm_backward(z, x, z, h, post_weight=w, pre_weight=w)
    assert not g["dpost_weight"].any() and not g["dpre_weight"].any()


def test_graph():
    """Captured passes, replayed with new inputs and a new offset, beside the eager ones."""
    dev = need_gpu()
    c = Case(dev, 130, 513, BF, BF, BF, F32, True, 1, True, 0.2, seed=2)

    def both():
        z, h = block_norm(c.x, c.y, **c.kw)
        return [z, h] + list(block_norm_backward(z, c.y, c.dz, c.dh, **c.kw).values())
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(3):
        c.kw["rng"].add_(i)
        c.x.mul_(1.5)
        want = [t.clone() for t in both()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_refusals():
    dev = need_gpu()
    x = torch.zeros((6, 64), dtype=BF, device=dev)
    w = torch.ones(64, dtype=BF, device=dev)
    for kw in (dict(), dict(gate=torch.ones((4, 64), dtype=BF, device=dev)), dict(post_weight=w.float(), pre_weight=w),
               dict(post_weight=w[:32]), dict(dropout=1.0), dict(dropout=0.5), dict(dropout=-0.1)):
        with pytest.raises(ValueError):
            block_norm(x, None if not kw else x.clone(), **kw)
    with pytest.raises(ValueError):
        block_norm(x, x[:, :32], post_weight=w)
    with pytest.raises(ValueError):
        block_norm(x.half(), x, post_weight=w)
    with pytest.raises(ValueError):
        block_norm(x.t(), None, pre_weight=w)
    with pytest.raises(ValueError):
        block_norm_backward(x, x, x, None, pre_weight=w)
    narrow = torch.zeros((6, 7), dtype=BF, device=dev)
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        block_norm(narrow, None, pre_weight=torch.ones(7, dtype=BF, device=dev))


def test_scale_of_a_tensor_is_read_at_each_call():
    dev = need_gpu()
    x = torch.randn((4, 64), generator=torch.Generator().manual_seed(1)).to(dev)
    y = torch.randn((4, 64), generator=torch.Generator().manual_seed(2)).to(dev)
    scale = torch.tensor(1.0)
    one, _ = block_norm(x, y, scale=scale)
    scale.fill_(2.0)
    two, _ = block_norm(x, y, scale=scale)
    assert torch.equal(one, x + y)
    assert torch.equal(two, torch.addcmul(x.double(), y.double(), torch.tensor(2.0, dtype=torch.float64, device=dev)).float())
