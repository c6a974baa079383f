"""The layer as a block of a model: norms, layer, gate, dropout and residual sum
together, forward and backward, against the whole block in fp64 differentiated by
torch, with the choice of experts that the GPU made.

Bound: each bf16 rounding on the way (h, the expert's h, its rows, out; in the
backward out's gradient, the replayed a, h, dy and da) moves what it rounds by at most
half a step, 2^-9, and by 2^-9 / sqrt(3) of its RMS.  Six of them that add linearly
give 6.8e-3: RMS(err) <= 2^-7 RMS.
"""

import pytest
import torch

from mixture_experts_layer_counts_amd import MoEBackward, MoELayer, prepare_backward, router_for, shape_for
from tests._gpu import need_gpu, say

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Block:
    def __init__(self, dev, T, D=192, I=128, E=12, k=3, Is=64, seed=0, stream=torch.float32):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape, std=1.0, add=0.0, dt=torch.bfloat16):
            return (torch.randn(shape, generator=g) * std + add).to(dt).to(dev)
        self.T, self.D, self.k = T, D, k
        self.x = rand(T, D, dt=stream)
        self.w_router = rand(E, D, std=D ** -0.5)
        self.w = {"w_gate": rand(E, I, D, std=D ** -0.5), "w_up": rand(E, I, D, std=D ** -0.5),
                  "w_down": rand(E, D, I, std=I ** -0.5), "ws_gate": rand(Is, D, std=D ** -0.5),
                  "ws_up": rand(Is, D, std=D ** -0.5), "ws_down": rand(D, Is, std=Is ** -0.5)}
        self.n = {"pre_weight": rand(D, std=0.2, add=1.0), "post_weight": rand(D, std=0.2, add=1.0),
                  "gate": rand(2, D), "next_weight": rand(D, std=0.2, add=1.0)}
        self.layer = MoELayer(shape_for(T, D, I, E, k, I_shared=Is), device=dev)
        self.rng = torch.tensor([77, 5], dtype=torch.int64, device=dev)

    def reference(self, idx, keep, p, kind, scale):
        """(leaves, z, h_next) in fp64, the experts as chosen."""
        v = {n: t.double().requires_grad_() for n, t in
             {"x": self.x, "w_router": self.w_router, **self.w, **self.n}.items()}

        def norm(t, w):
            return t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * w

        def ffn(t, g, u, d):
            a = t @ g.T
            return (a * torch.sigmoid(a) * (t @ u.T)) @ d.T
        h = norm(v["x"], v["pre_weight"])
        logits = h @ v["w_router"].T
        s = torch.sigmoid(logits) if kind == "sigmoid" else torch.softmax(logits, -1)
        gates = torch.gather(s, 1, idx.long())
        gates = gates / gates.sum(1, keepdim=True)
        out = ffn(h, v["ws_gate"], v["ws_up"], v["ws_down"])
        rows = []
        for t in range(self.T):
            rows.append(sum(gates[t, j] * ffn(h[t:t + 1], v["w_gate"][e], v["w_up"][e], v["w_down"][e])[0]
                            for j, e in enumerate(idx[t].tolist())))
        out = out + torch.stack(rows)
        y = norm(out, v["post_weight"]) * v["gate"].repeat_interleave(self.T // 2, 0) * scale
        if keep is not None:
            y = torch.where(keep, y / (1 - p), 0.0)
        z = v["x"] + y
        return v, z, norm(z, v["next_weight"])


def off(got, want):
    return float((got.double() - want).square().mean().sqrt() / want.square().mean().sqrt())


def kept(block, p):
    """Dropout's mask, from a call on ones."""
    from mixture_experts_layer_counts_amd import block_norm
    if not p:
        return None
    x = torch.zeros((block.T, block.D), device=block.x.device)
    z, _ = block_norm(x, torch.ones_like(x), dropout=p, rng=block.rng)
    return z != 0


@pytest.mark.parametrize("T,train,p,router", [
    (2, False, 0.0, None), (64, False, 0.1, dict(score="sigmoid")), (64, True, 0.1, None),
    (66, False, 0.0, dict(score="sigmoid")), (130, True, 0.0, dict(score="softmax")),
])
def test_forward_and_backward(T, train, p, router):
    dev = need_gpu()
    say("block", T, train, p, router)
    b = Block(dev, T, seed=T)
    kw = dict(b.n, scale=0.5, dropout=p, rng=b.rng if p else None, router=router_for(**router) if router else None)
    r = b.layer.block(b.x, b.w_router, b.w, train=train, **kw)
    assert ("counts" in r) == (train or T > 64)  # few tokens: one launch, no schedule
    assert b.layer.device_error() == 0
    v, z, h_next = b.reference(r["idx"], kept(b, p), p, (router or {}).get("score", "softmax"), 0.5)
    say("  z", off(r["z"] - b.x, (z - v["x"]).detach()), "h_next", off(r["h_next"], h_next.detach()))
    assert off(r["z"] - b.x, (z - v["x"]).detach()) <= 2.0 ** -7
    assert off(r["h_next"], h_next.detach()) <= 2.0 ** -7
    if not train:
        return
    g = torch.Generator().manual_seed(1)
    dz = torch.randn((T, b.D), generator=g).to(dev)
    dh = torch.randn((T, b.D), generator=g).to(dev).to(torch.bfloat16)
    bw = prepare_backward(b.layer.shape, b.w, b.w_router)
    back = MoEBackward(b.layer.shape, device=dev)
    got = back.block(bw, b.x, r, b.layer.routed_rows(), dz, dh, **kw)
    assert back.device_error() == 0
    ((z * dz.double()).sum() + (h_next * dh.double()).sum()).backward()
    names = {"dx": "x", "dpre_weight": "pre_weight", "dpost_weight": "post_weight", "dgate": "gate",
             "dnext_weight": "next_weight", "dw_router": "w_router", "dw_gate": "w_gate", "dw_up": "w_up",
             "dw_down": "w_down", "dws_gate": "ws_gate", "dws_up": "ws_up", "dws_down": "ws_down"}
    for n, m in names.items():
        err = off(got[n], v[m].grad)
        say("  ", n, err)
        # weight gradients: products of rounded factors, and rounded themselves once more
        assert err <= 2.0 ** -6 if n.startswith("dw") else err <= 2.0 ** -7, n


def test_a_stream_of_blocks():
    """Two blocks in a row, the second on what the first prepared, captured and replayed on another stream."""
    dev = need_gpu()
    b = Block(dev, 4, seed=9, stream=torch.bfloat16)

    def two():
        r = b.layer.block(b.x, b.w_router, b.w, **b.n, scale=0.5)
        q = b.layer.block(r["z"], b.w_router, b.w, **b.n, scale=0.5)
        return r["z"], q["z"], q["h_next"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        two()
        two()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = two()
    for i in range(4):
        b.x.mul_(-1.25)
        want = [t.clone() for t in two()]
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(got, want):
            assert torch.equal(a, c)
    assert b.layer.device_error() == 0
