"""Calls of several shapes on one workspace, in stream order: moe_few for different token counts, widths and
precisions, and moe_forward of a larger shape between them, give the bits that they give on workspaces of their own."""

import ctypes

import pytest
import torch

from mixture_experts_layer_counts_amd import MoELayer, shape_for
from tests._gpu import need_gpu, say
from tests.test_gpu_few import Case

pytestmark = pytest.mark.gpu


def same(a, b):
    return all(torch.equal(a[n], b[n]) for n in ("logits", "idx", "gate", "out", "out32"))


def test_one_workspace_for_several_shapes():
    dev = need_gpu()
    cases = [Case(dev, 4, 512, 192, 40, 4, seed=1), Case(dev, 5, 512, 192, 40, 4, seed=2, tiled=True),
             Case(dev, 64, 512, 192, 40, 4, seed=3), Case(dev, 1, 256, 64, 9, 2, seed=4),
             Case(dev, 7, 384, 256, 20, 4, Is=128, prec="mxfp8", sprec="mxfp8", seed=5),
             Case(dev, 16, 2048, 64, 300, 16, seed=6)]
    large = Case(dev, 700, 512, 192, 40, 4, seed=7)
    want = [c.layer.few(c.x, c.w_router, c.weights) for c in cases]
    want_large = large.layer(large.x, large.w_router, large.weights)
    torch.cuda.synchronize()
    layers = [c.layer for c in cases] + [large.layer]
    # bytes of any kind, then one initialisation, by the smallest shape
    ws = torch.full((max(l.ws_bytes for l in layers),), 0xA5, dtype=torch.uint8, device=dev)
    for l in layers:
        l.ws, l.ws_bytes = ws, ws.numel()
    assert cases[3].layer.lib.moe_workspace_init(ctypes.byref(cases[3].layer.shape), ctypes.c_void_p(ws.data_ptr()),
                                                 ws.numel(), None) == 0
    for turn in range(4):
        for i in range(len(cases)):
            j = (i * (turn + 1) + turn) % len(cases) if turn % 2 else i
            c = cases[j]
            say("shared workspace", turn, j)
            assert same(c.layer.few(c.x, c.w_router, c.weights), want[j])
        r = large.layer(large.x, large.w_router, large.weights)
        assert same(r, want_large)
    assert large.layer.device_error() == 0


def test_graphs_of_two_shapes_on_one_workspace():
    """Captured calls of two shapes, replayed in turn in stream order on one workspace, beside eager ones."""
    dev = need_gpu()
    a, b = Case(dev, 3, 512, 192, 40, 4, seed=8), Case(dev, 33, 384, 128, 24, 3, seed=9)
    ws = torch.zeros(max(a.layer.ws_bytes, b.layer.ws_bytes), dtype=torch.uint8, device=dev)
    for c in (a, b):
        c.layer.ws, c.layer.ws_bytes = ws, ws.numel()
    assert a.layer.lib.moe_workspace_init(ctypes.byref(a.layer.shape), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                          None) == 0
    torch.cuda.synchronize()
    graphs, got = [], []
    for c in (a, b):
        c.layer.few(c.x, c.w_router, c.weights)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(c.layer.few(c.x, c.w_router, c.weights))
        graphs.append(g)
    for i in range(5):
        a.x.mul_(-1.25)
        b.x.add_(0.125)
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        want = [c.layer.few(c.x, c.w_router, c.weights) for c in (a, b)]
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])
    assert a.layer.device_error() == 0


def test_block_of_no_rows():
    dev = need_gpu()
    layer = MoELayer(shape_for(0, 128, 64, 8, 2), device=dev)
    c = Case(dev, 2, 128, 64, 8, 2)
    w = torch.ones(128, dtype=torch.bfloat16, device=dev)
    r = layer.block(c.x[:0], c.w_router, c.weights, w, post_weight=w, next_weight=w)
    assert r["z"].shape == (0, 128) and r["h_next"].shape == (0, 128) and r["out"].shape == (0, 128)
