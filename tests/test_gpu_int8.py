"""GPU parity of the 8-bit integer operators: moe_quantize_int8 and
moe_matmul_int8 bit for bit, and the int8 experts of moe_forward.

Quotients, sums and the two scalings are defined to the bit, so the first two
are compared for equality.  A layer's output is not: SiLU is approximated (to
about 2^-20) before h is quantised, so a value of h within 127 2^-20 of a
border between two integers may fall on its other side.  That is below 2.5e-4
of the values, half a value a row at I = 2048; 8 such steps a row are allowed,
each of m_h / 127 times the largest weight of the channel.  The routed rows are
stored bf16, half a step 2^-8 of the value, and the rest is fp32: 2^-20.
"""

import numpy as np
import pytest
import torch

import synth
from mixture_experts_layer_counts_amd import (MoELayer, linear_int8, matmul_int8, quantize_int8, router_for, shape_for,
                                              tile_int8)
from oracle import int8
from tests._gpu import mx_shared_weights_dev, mx_weights_dev, need_gpu, say, to_dev

pytestmark = pytest.mark.gpu


def rows_with_ties(rows, K, dtype, seed):
    """Normal rows; some with entries whose quotient 127 v / m is half an integer."""
    v = torch.randn((rows, K), generator=torch.Generator().manual_seed(seed)).to(dtype)
    for r in range(0, rows, 3):
        v[r] = torch.where(v[r].abs() > 2.0, v[r], (v[r] * 16).round() / 16).clamp(-4, 4)
        v[r, -1] = 4.0 if r % 2 else 127.0 / 32
    return v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (5, 128), (7, 130), (9, 1001), (4, 2048), (2, 7168), (3, 8200),
                                    (2, 40001), (300, 256)])
def test_quantize_int8(rows, K, dtype):
    dev = need_gpu()
    say("quantize_int8", rows, K, dtype)
    v = rows_with_ties(rows, K, dtype, K)
    q, s = quantize_int8(v.to(dev))
    wq, _ = int8.quantize(v.double().numpy())
    Kp = (K + 127) // 128 * 128
    assert q.shape == (rows, Kp)
    got = q.cpu().numpy()
    assert np.array_equal(got[:, :K], wq) and np.all(got[:, K:] == 0)
    m = np.abs(v.float().numpy()).max(axis=1)
    assert np.array_equal(s.cpu().numpy(), m / np.float32(127))


def test_quantize_int8_special_rows():
    dev = need_gpu()
    say("quantize_int8 special")
    v = torch.zeros((8, 200))
    v[1, 3], v[2, 5], v[3, 199] = float("inf"), float("nan"), -float("inf")
    v[4, 0], v[4, 1] = torch.finfo(torch.float32).max, torch.finfo(torch.float32).min / 2
    v[5, 0], v[5, 1] = 1e-45, -1e-45  # the smallest numbers
    v[6, 0], v[6, 1] = 1.0, 2.0 ** -120
    v[7, ::2] = -0.0
    # near the largest floats, values on either side of a half, and the half itself
    top = torch.finfo(torch.float32).max
    big = torch.zeros((1, 200))
    big[0, 0] = top
    big[0, 1:9] = torch.tensor([top / 2, top / 254, 3 * (top / 254), -5 * (top / 254), top / 127, -top / 2,
                                7 * (top / 254), 0.0])
    qb, _ = quantize_int8(big.to(dev))
    assert np.array_equal(qb.cpu().numpy()[:, :200], int8.quantize(big.double().numpy())[0])
    q, s = (t.cpu() for t in quantize_int8(v.to(dev)))
    assert torch.isnan(s[1:4]).all() and (q[1:4] == 0).all()
    assert (q[0] == 0).all() and s[0] == 0 and (q[7] == 0).all() and s[7] == 0
    assert q[4, :2].tolist() == [127, -64] and q[5, :2].tolist() == [127, -127] and q[6, :2].tolist() == [127, 0]
    # a row that is not finite gives NaN, and only in its own row
    w = torch.ones((16, 256), dtype=torch.int8, device=dev)
    out = matmul_int8(q.to(dev), s.to(dev), w, torch.ones(16, device=dev)).cpu()
    assert torch.isnan(out[1:4]).all() and torch.isfinite(out[[0, 5, 6, 7]]).all()


def reference(q, s, wq, ws, dtype):
    acc = (q.double() @ wq.double().T).float()  # exact integers, rounded to fp32 once
    return ((acc * s[:, None]) * ws[None, :]).to(dtype)


MATS = [(1, 1, 128), (1, 2048, 7168), (2, 17, 256), (15, 33, 384), (16, 64, 128), (17, 1001, 1536), (32, 130, 2048),
        (33, 257, 640), (64, 512, 1024), (100, 96, 128), (255, 300, 256), (257, 511, 384), (777, 1001, 1536),
        (1024, 768, 2048), (513, 8, 65536),
        # sizes for which the product takes tiles of 64, 128, 256 and 320 rows
        (777, 2048, 128), (777, 7168, 256), (2050, 7168, 128), (2400, 8190, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", MATS, ids=lambda v: str(v))
def test_matmul_int8(M, N, K, dtype):
    dev = need_gpu()
    say("matmul_int8", M, N, K, dtype)
    gen = torch.Generator().manual_seed(M + N)
    q = torch.randint(-127, 128, (M, K), generator=gen, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=gen, dtype=torch.int8)
    if M > 1:
        q[1], w[0] = 127, 127  # the largest sum there is
    s, ws = torch.rand(M, generator=gen), torch.rand(N, generator=gen) - 0.5
    got = matmul_int8(q.to(dev), s.to(dev), w.to(dev), ws.to(dev), out_dtype=dtype).cpu()
    assert torch.equal(got, reference(q, s, w, ws, dtype))


# Resident workgroups that walk on from a tile whose last rows do not fill an 8-row piece of the output: more
# items than workgroups, in tiles of 256 rows (the first seven and the last) and of 320, which end in 1 to 5 rows mod 8.
HANDOVERS = [(2905, 7168, 128), (2969, 7168, 128), (2970, 7168, 512), (2972, 7168, 128), (3002, 7168, 256),
             (5276, 4096, 128), (8187, 4096, 128), (4609, 7168, 128), (4610, 7168, 384), (8195, 4096, 256),
             (4605, 7168, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", HANDOVERS, ids=lambda v: str(v))
def test_matmul_int8_of_ragged_tiles_between_others(M, N, K, dtype):
    dev = need_gpu()
    say("matmul_int8 handover", M, N, K, dtype)
    gen = torch.Generator().manual_seed(M + K)
    q = torch.randint(-127, 128, (M, K), generator=gen, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=gen, dtype=torch.int8)
    s, ws = torch.rand(M, generator=gen), torch.rand(N, generator=gen) - 0.5
    args = [t.to(dev) for t in (q, s, w, ws)]
    # sums below 2^24 (K <= 512): an fp32 product of the integers is exact
    want = ((args[0].float() @ args[2].float().T) * args[1][:, None] * args[3][None, :]).to(dtype)
    for rep in range(3):
        assert torch.equal(matmul_int8(*args, out_dtype=dtype), want), rep


def test_matmul_int8_writes_only_its_rows():
    # a result inside a larger buffer of the allocator stays inside it: rows past M keep their bytes
    dev = need_gpu()
    from mixture_experts_layer_counts_amd import _lib
    lib = _lib.load()
    for M, N in ((5, 37), (40, 129), (300, 257)):
        q = torch.ones((M, 128), dtype=torch.int8, device=dev)
        w = torch.ones((N, 128), dtype=torch.int8, device=dev)
        one_m, one_n = torch.ones(M, device=dev), torch.ones(N, device=dev)
        buf = torch.full((M * N + 512,), -7.0, device=dev)
        assert lib.moe_matmul_int8(q.data_ptr(), one_m.data_ptr(), M, w.data_ptr(), one_n.data_ptr(), N, 128,
                                   buf.data_ptr(), 1, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert (buf[:M * N] == 128).all() and (buf[M * N:] == -7).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lead,K,N", [((1,), 100, 7), ((2, 9), 1500, 301), ((130,), 7168, 256)])
def test_linear_int8(lead, K, N, dtype):
    dev = need_gpu()
    say("linear_int8", lead, K, N)
    gen = torch.Generator().manual_seed(N)
    x = torch.randn(lead + (K,), generator=gen).to(dtype)
    wq, ws = quantize_int8((torch.randn((N, K), generator=gen) / K ** 0.5).to(dev))
    for out_dtype in (None, torch.float32):
        got = linear_int8(x.to(dev), wq, ws, out_dtype)
        q, _ = int8.quantize(x.double().numpy().reshape(-1, K))
        s = x.float().abs().amax(dim=-1).reshape(-1) / 127.0
        want = reference(torch.from_numpy(q), s, wq.cpu()[:, :K], ws.cpu(), dtype if out_dtype is None else out_dtype)
        assert got.shape == lead + (N,) and torch.equal(got.cpu().reshape(-1, N), want)
    empty = linear_int8(torch.empty((0, K), dtype=dtype, device=dev), wq, ws)
    assert empty.shape == (0, N)


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------
def quantised(inp, dev, routed=True, shared=True, tiled=False):
    w = {}
    for n in ("gate", "up", "down"):
        if routed:
            w["q_" + n], w["s_" + n] = quantize_int8(inp["w_" + n].to(dev))
            if tiled:
                w["q_" + n] = tile_int8(w["q_" + n])
        else:
            w["w_" + n] = inp["w_" + n].to(dev)
        if shared:
            w["qs_" + n], w["ss_" + n] = quantize_int8(inp["ws_" + n].to(dev))
        else:
            w["ws_" + n] = inp["ws_" + n].to(dev)
    return w


def oracle(w, inp, idx, gate, routed=True, shared=True):
    """(out, bound) in fp64 for the layer with int8 routed and shared experts."""
    x = inp["x"].double().numpy()
    wq = {}
    for n in ("gate", "up", "down"):
        wq["q_" + n], wq["s_" + n] = int8.quantize(inp["w_" + n].double().numpy())
        wq["qs_" + n], wq["ss_" + n] = int8.quantize(inp["ws_" + n].double().numpy())
    out, tol = np.zeros((w.T, w.D)), np.zeros((w.T, w.D))

    def add(rows, xr, g, prefix, e, step):
        y, m = int8.ffn(xr, wq, prefix, e)
        q, s = wq[f"q{prefix}_down"], wq[f"s{prefix}_down"]
        big = np.abs(q if e is None else q[e]).max(axis=1) * (s if e is None else s[e])
        out[rows] += g[:, None] * y
        tol[rows] += np.abs(g)[:, None] * (step * np.abs(y) + 8 * (m / 127)[:, None] * big[None, :])
    for e in range(w.E):
        t, slot = np.nonzero(idx == e)
        if len(t):
            add(t, x[t], gate[t, slot].astype(np.float64), "", e, 2.0 ** -8 + 2.0 ** -20)
    add(np.arange(w.T), x, np.ones(w.T), "s", None, 2.0 ** -20)
    return out, tol + 2.0 ** -20 * np.abs(out)


LAYERS = [  # workload, minibatch, ring
    (synth.Workload("one", T=1, D=256, I=128, E=8, k=2, I_shared=128, seed=1, routing="gaussian"), None, None),
    (synth.Workload("few", T=5, D=512, I=256, E=64, k=8, I_shared=384, seed=2, routing="gaussian"), None, None),
    (synth.Workload("ragged", T=300, D=256, I=384, E=16, k=4, I_shared=128, seed=7, routing="gaussian"), None, None),
    (synth.Workload("ragged", T=300, D=256, I=384, E=16, k=4, I_shared=128, seed=7, routing="gaussian"), 256, 512),
    (synth.Workload("skewed", T=1100, D=384, I=128, E=24, k=6, I_shared=256, seed=8, routing="zipf"), None, None),
    # 25, 64 and 200 rows an expert: tiles of 64, 192 and 320 rows (those above take 32 and 128)
    (synth.Workload("rows25", T=100, D=256, I=256, E=16, k=4, I_shared=128, seed=10, routing="gaussian"), None, None),
    (synth.Workload("rows64", T=1024, D=128, I=1280, E=128, k=8, I_shared=128, seed=11, routing="gaussian"), None,
     None),
    (synth.Workload("rows200", T=4800, D=128, I=1024, E=96, k=4, I_shared=128, seed=12, routing="zipf"), None, None),
    # shared experts whose up/gate takes tiles of 64, 128, 256 and 320 rows
    (synth.Workload("shared64", T=777, D=128, I=128, E=4, k=1, I_shared=2048, seed=15, routing="gaussian"), None, None),
    (synth.Workload("shared128", T=777, D=128, I=128, E=4, k=1, I_shared=7168, seed=16, routing="gaussian"), None,
     None),
    (synth.Workload("shared256", T=2050, D=128, I=128, E=4, k=1, I_shared=7168, seed=17, routing="gaussian"), None,
     None),
    (synth.Workload("shared320", T=2400, D=128, I=128, E=4, k=1, I_shared=8192, seed=18, routing="gaussian"), None,
     None),
    # a few large experts: items drawn from the queues, at tiles of 64, 128 and 320 rows
    (synth.Workload("zipf64", T=600, D=128, I=512, E=64, k=4, I_shared=128, seed=19, routing="zipf"), None, None),
    (synth.Workload("zipf128", T=1700, D=256, I=384, E=64, k=4, I_shared=128, seed=20, routing="zipf"), None, None),
    (synth.Workload("zipf320", T=6100, D=128, I=1152, E=96, k=4, I_shared=128, seed=22, routing="zipf"), None, None),
    (synth.Workload("single", T=700, D=128, I=128, E=1, k=1, I_shared=128, seed=9, routing="gaussian"), None, None),
]


def make(w, dev, b=None, C=None, tiled=False, precision="int8", shared="int8"):
    return MoELayer(shape_for(w.T, w.D, w.I, w.E, w.k, I_shared=w.I_shared, minibatch_rows=b, ring_rows=C,
                              precision=precision, shared_precision=shared, weights_tiled=tiled), device=dev)


@pytest.mark.parametrize("w,b,C", LAYERS, ids=[f"{c[0].name}-{c[1]}" for c in LAYERS])
def test_int8_layer_parity(w, b, C):
    dev = need_gpu()
    say("int8 layer", w, b, C)
    inp = synth.make_inputs(w)
    x, lg = inp["x"].to(dev), inp["logits"].to(dev)
    outs = []
    for tiled in (False, True):
        m = make(w, dev, b, C, tiled)
        r = m(x, None, quantised(inp, dev, tiled=tiled), logits=lg)
        torch.cuda.synchronize()
        assert m.device_error() == 0
        outs.append(r["out32"])
    assert torch.equal(outs[0], outs[1])  # the layout of the weights changes no bit
    want, tol = oracle(w, inp, r["idx"].cpu().numpy(), r["gate"].cpu().numpy())
    err = np.abs(r["out32"].cpu().numpy() - want)
    say("   max err / bound", (err / tol).max())
    assert np.all(err <= tol)
    assert torch.equal(r["out"], r["out32"].to(torch.bfloat16))


def test_int8_layer_is_the_same_for_every_minibatch():
    dev = need_gpu()
    w = synth.Workload("ragged", T=300, D=256, I=384, E=16, k=4, I_shared=128, seed=7, routing="gaussian")
    inp = synth.make_inputs(w)
    x, lg = inp["x"].to(dev), inp["logits"].to(dev)
    wd = quantised(inp, dev)
    want = make(w, dev)(x, None, wd, logits=lg)["out32"]
    for b, C in ((1, 1), (7, 7), (64, 128), (1000, 2000)):
        got = make(w, dev, b, C)(x, None, wd, logits=lg)["out32"]
        assert torch.equal(got, want), (b, C)


def random_layer(dev, T, D, I, E, k, seed):
    """Weights drawn as int8 (no quantiser), routes and gates, all on the GPU."""
    gen = torch.Generator(device=dev).manual_seed(seed)
    w = {}
    for n, (a, b) in (("gate", (I, D)), ("up", (I, D)), ("down", (D, I))):
        w["q_" + n] = torch.randint(-60, 61, (E, a, b), dtype=torch.int8, device=dev, generator=gen)
        w["qs_" + n] = torch.randint(-60, 61, (a, b), dtype=torch.int8, device=dev, generator=gen)
        w["s_" + n] = 1e-3 * torch.rand((E, a), device=dev, generator=gen)
        w["ss_" + n] = 1e-3 * torch.rand(a, device=dev, generator=gen)
    x = torch.randn((T, D), device=dev, generator=gen).to(torch.bfloat16)
    idx = torch.rand((T, E), device=dev, generator=gen).topk(k, dim=1).indices.to(torch.int32).contiguous()
    return w, x, idx, torch.rand((T, k), device=dev, generator=gen)


def test_int8_mid_layer_is_the_same_for_every_tile_height_and_on_every_run():
    # 256 rows an expert (320-row tiles, a resident workgroup walks several items), 64 and 8 of
    # them in a minibatch (128-row tiles, and 64-row ones): the integer sums give the same bits
    dev = need_gpu()
    T, D, I, E, k = 4096, 2048, 768, 128, 8
    w, x, idx, gate = random_layer(dev, T, D, I, E, k, 5)
    want = None
    for b in (None, None, 8192, 1024, 512, None):
        say("int8 mid, minibatch", b)
        m = MoELayer(shape_for(T, D, I, E, k, minibatch_rows=b, precision="int8", shared_precision="int8"), device=dev)
        _, got = m.forward(w, x, x, gate, m.schedule(idx))
        torch.cuda.synchronize()
        want = got if want is None else want
        assert torch.equal(got, want), b


@pytest.mark.parametrize("D,I,E,per", [
    # 320-, 192-, 128- and 64-row tiles of the routed products, several items a workgroup
    (2048, 1152, 96, 196), (2048, 2048, 64, 145), (2048, 1408, 64, 101), (2048, 1152, 128, 21)])
def test_int8_layer_of_ragged_experts(D, I, E, per):
    # experts of per + 1, per + 2, ... per + 8 rows in turn, so that tiles end in every count of rows mod 8: the bits
    # of minibatches that take the few-rows kernel
    dev = need_gpu()
    say("int8 ragged experts", D, I, E, per)
    ids = torch.repeat_interleave(torch.arange(E), torch.tensor([per + 1 + e % 8 for e in range(E)]))
    T = len(ids)
    w, x, _, gate = random_layer(dev, T, D, I, E, 1, 23)
    ids = ids[torch.randperm(T, generator=torch.Generator().manual_seed(T))]
    idx = ids.to(torch.int32).view(T, 1).to(dev)
    kw = dict(precision="int8", shared_precision="int8")
    small = MoELayer(shape_for(T, D, I, E, 1, minibatch_rows=4 * E, **kw), device=dev)
    small.forward(w, x, x, gate, small.schedule(idx))
    want = small.routed_rows().clone()
    m = MoELayer(shape_for(T, D, I, E, 1, **kw), device=dev)
    for rep in range(3):
        m.routed_rows().zero_()
        m.forward(w, x, x, gate, m.schedule(idx))
        assert torch.equal(m.routed_rows(), want), rep
    assert m.device_error() == 0


def test_int8_layer_with_rows_that_the_table_drops():
    # a table of the caller's own, with entries outside the routes: those rows write nothing, the others keep their bits
    dev = need_gpu()
    D, I, E, T = 2048, 1152, 96, 19248
    say("int8 dropped rows", D, I, E)
    w, x, _, gate = random_layer(dev, T, D, I, E, 1, 37)
    idx = (torch.arange(T, device=dev) % E).to(torch.int32).view(T, 1)
    m = MoELayer(shape_for(T, D, I, E, 1, precision="int8", shared_precision="int8"), device=dev)
    sched = m.schedule(idx)
    m.forward(w, x, x, gate, sched)
    want = m.routed_rows().clone()
    p = torch.arange(T, device=dev)
    drop = (p % 24 >= 8) | (p % 7 == 3)
    routes = sched["sched"][drop].long()
    sched["sched"][drop] = torch.where(p[drop] % 2 == 0, -1, T + 5).to(torch.int32)
    want[routes] = -3.0
    for rep in range(3):
        m.routed_rows().fill_(-3.0)
        m.forward(w, x, x, gate, sched)
        assert torch.equal(m.routed_rows(), want), rep


@pytest.mark.parametrize("T,b", [(2, None), (40, None), (300, None), (300, 128)])
def test_int8_layer_flags_a_table_with_entries_out_of_range(T, b):
    # as the bf16 and MXFP8 layers do: no route is dropped without the error bit
    dev = need_gpu()
    say("int8 bad table", T, b)
    w = synth.Workload("table", T=T, D=256, I=128, E=8, k=2, I_shared=128, seed=41, routing="gaussian")
    inp = synth.make_inputs(w)
    x, wd = inp["x"].to(dev), quantised(inp, dev)
    for bad in (-1, T * w.k):
        m = make(w, dev, b=b)
        _, idx, gate = m.route(None, None, inp["logits"].to(dev))
        sched = m.schedule(idx)
        m.forward(wd, x, x, gate, sched)
        assert m.device_error() == 0
        sched["sched"][T * w.k - 1] = bad
        m.forward(wd, x, x, gate, sched)
        assert m.device_error() == 0x1, bad


@pytest.mark.parametrize("T,I_shared", [(2561, 4096), (2570, 4096), (5123, 2048), (4098, 4096), (4107, 4096)])
def test_int8_shared_expert_of_ragged_tiles(T, I_shared):
    # 256- and 320-row SwiGLU tiles, several items a workgroup: the bits of 32 tokens at a time
    dev = need_gpu()
    say("int8 shared ragged", T, I_shared)
    D = 128
    gen = torch.Generator(device=dev).manual_seed(T)
    w, x, idx, gate = random_layer(dev, T, D, 128, 2, 1, 29)
    for n, (a, b) in (("gate", (I_shared, D)), ("up", (I_shared, D)), ("down", (D, I_shared))):
        w["qs_" + n] = torch.randint(-60, 61, (a, b), dtype=torch.int8, device=dev, generator=gen)
        w["ss_" + n] = 1e-3 * torch.rand(a, device=dev, generator=gen)
    gate = torch.zeros_like(gate)  # the routed part adds nothing
    kw = dict(I_shared=I_shared, precision="int8", shared_precision="int8")
    few = MoELayer(shape_for(32, D, 128, 2, 1, **kw), device=dev)
    want = []
    for t in range(0, T, 32):
        rows = torch.arange(t, t + 32, device=dev).clamp(max=T - 1)
        xs, ids, gs = x[rows], idx[rows], gate[rows]
        want.append(few.forward(w, xs, xs, gs, few.schedule(ids))[1])
    want = torch.cat(want)[:T]
    m = MoELayer(shape_for(T, D, 128, 2, 1, **kw), device=dev)
    for rep in range(3):
        assert torch.equal(m.forward(w, x, x, gate, m.schedule(idx))[1], want), rep
    assert m.device_error() == 0


@pytest.mark.parametrize("hot", ["one", "two", "most"])
def test_int8_hot_experts(hot):
    # routes that leave most experts, and most XCDs' shares, without rows: the bits of small minibatches, on every
    # run, and in a graph
    dev = need_gpu()
    T, D, I, E, k = 3000, 256, 640, 40, 2
    say("int8 hot experts", hot)
    w, x, idx, gate = random_layer(dev, T, D, I, E, k, 17)
    if hot == "one":
        idx[:] = torch.tensor([7, 8], dtype=torch.int32, device=dev)  # two experts in all
    elif hot == "two":
        idx[:, 0], idx[:, 1] = 0, (torch.arange(T, device=dev) % 2 + E - 2).to(torch.int32)
    else:
        idx[: T - 200] = torch.tensor([20, 3], dtype=torch.int32, device=dev)
    kw = dict(precision="int8", shared_precision="int8")
    small = MoELayer(shape_for(T, D, I, E, k, minibatch_rows=96, ring_rows=192, **kw), device=dev)
    want = small.forward(w, x, x, gate, small.schedule(idx))[1]
    m = MoELayer(shape_for(T, D, I, E, k, **kw), device=dev)
    for _ in range(3):
        assert torch.equal(m.forward(w, x, x, gate, m.schedule(idx))[1], want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = m.forward(w, x, x, gate, m.schedule(idx))[1]
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert torch.equal(m.forward(w, x, x, gate, m.schedule(idx))[1], want)
    assert m.device_error() == 0 and small.device_error() == 0


def test_int8_layers_on_two_streams_at_once():
    dev = need_gpu()
    T, D, I, E, k = 200, 512, 256, 32, 4
    layers, streams, inputs, want = [], [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for i in range(2):
        inputs.append(random_layer(dev, T, D, I, E, k, 30 + i))
        layers.append(MoELayer(shape_for(T, D, I, E, k, precision="int8", shared_precision="int8"), device=dev))
        w, x, idx, gate = inputs[i]
        want.append(layers[i].forward(w, x, x, gate, layers[i].schedule(idx))[1].clone())
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            w, x, idx, gate = inputs[i]
            with torch.cuda.stream(streams[i]):
                got[i] = layers[i].forward(w, x, x, gate, layers[i].schedule(idx))[1]
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i])


@pytest.mark.parametrize("routed,shared", [(True, False), (False, True)])
def test_int8_for_one_kind_of_expert(routed, shared):
    # bf16 experts beside int8 ones: the int8 part of the result is the same bits as in the all-int8 layer
    dev = need_gpu()
    w = synth.Workload("mixed", T=130, D=256, I=128, E=8, k=2, I_shared=128, seed=4, routing="gaussian")
    say("int8 mixed", routed, shared)
    inp = synth.make_inputs(w)
    x, lg = inp["x"].to(dev), inp["logits"].to(dev)
    both = make(w, dev)
    rb = both(x, None, quantised(inp, dev), logits=lg)
    yb = both.routed_rows().clone()
    m = make(w, dev, precision="int8" if routed else "bf16", shared="int8" if shared else "bf16")
    r = m(x, None, quantised(inp, dev, routed, shared), logits=lg)
    y = m.routed_rows().clone()
    plain = make(w, dev, precision="bf16", shared="bf16")
    rp = plain(x, None, to_dev(inp, dev), logits=lg)
    if routed:
        assert torch.equal(y, yb)
    else:
        assert torch.equal(y, plain.routed_rows())
    # out32 = (sum of routed, in order) + shared: what is left of one is the other's
    g = r["gate"].double()
    def shared_part(res, rows):
        return res["out32"].double() - (g[:, :, None] * rows.double().view(w.T, w.k, w.D)).sum(1)
    other = shared_part(rb if shared else rp, yb if shared else plain.routed_rows())
    scale = r["out32"].abs().max().double()
    assert (shared_part(r, y) - other).abs().max() <= 2.0 ** -20 * scale


@pytest.mark.parametrize("T", [1, 130])
@pytest.mark.parametrize("routed", [True, False])
def test_int8_beside_mxfp8(routed, T):
    # int8 and MXFP8 experts in one layer: each part has the bits it has beside its own kind
    dev = need_gpu()
    w = synth.Workload("int8-mx", T=T, D=256, I=128, E=8, k=2, I_shared=128, seed=6, routing="gaussian")
    say("int8 beside mxfp8", routed, T)
    inp = synth.make_inputs(w)
    d = to_dev(inp, dev)
    x, lg = d["x"], d["logits"]
    weights = quantised(inp, dev, routed=routed, shared=not routed)
    mx = {**mx_weights_dev(d), **mx_shared_weights_dev(d)}
    weights = {n: v for n, v in weights.items() if not n.startswith("w")}
    weights.update({n: v for n, v in mx.items() if n not in weights})
    kinds = ("int8", "mxfp8") if routed else ("mxfp8", "int8")
    m = make(w, dev, precision=kinds[0], shared=kinds[1])
    r = m(x, None, weights, logits=lg)
    y = m.routed_rows().clone()
    ref_i8, ref_mx = make(w, dev), make(w, dev, precision="mxfp8", shared="mxfp8")
    ri, rm = ref_i8(x, None, quantised(inp, dev), logits=lg), ref_mx(x, None, mx, logits=lg)
    torch.cuda.synchronize()
    assert m.device_error() == 0
    yi, ym = ref_i8.routed_rows().clone(), ref_mx.routed_rows().clone()
    assert torch.equal(y, yi if routed else ym)
    g = r["gate"].double()

    def shared_part(res, rows):
        return res["out32"].double() - (g[:, :, None] * rows.double().view(w.T, w.k, w.D)).sum(1)
    other = shared_part(rm, ym) if routed else shared_part(ri, yi)
    assert (shared_part(r, y) - other).abs().max() <= 2.0 ** -20 * r["out32"].abs().max().double()


@pytest.mark.parametrize("K,N", [(100, 33), (1500, 301), (7168, 256), (20480, 48), (40960, 16), (65536, 16)])
def test_linear_int8_of_few_rows_is_the_same_as_of_many(K, N):
    # up to three rows that fit in LDS are quantised inside the product, more or longer ones before it
    dev = need_gpu()
    say("linear few rows", K, N)
    gen = torch.Generator().manual_seed(K)
    wq, ws = quantize_int8(torch.randn((N, K), generator=gen).to(dev))
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn((6, K), generator=gen).to(dtype).to(dev)
        x[4, 3] = float("nan")
        want = linear_int8(x, wq, ws, torch.float32)
        assert torch.isnan(want[4]).all()
        for M in (1, 2, 3, 4):
            for first in (0, 6 - M):
                got = linear_int8(x[first:first + M].clone(), wq, ws, torch.float32)
                assert torch.equal(got.view(torch.int32), want[first:first + M].view(torch.int32)), (dtype, M, first)


@pytest.mark.parametrize("M", [1, 2, 40])
def test_linear_int8_in_a_graph(M):
    # captured, replayed on new rows between eager calls on two streams
    dev = need_gpu()
    K, N = 1500, 776
    say("linear graph", M)
    gen = torch.Generator().manual_seed(M)
    wq, ws = quantize_int8(torch.randn((N, K), generator=gen).to(dev))
    x = torch.randn((M, K), generator=gen).to(torch.bfloat16).to(dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        linear_int8(x, wq, ws, out_dtype=torch.float32)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = linear_int8(x, wq, ws, out_dtype=torch.float32)
    for rep in range(3):
        x.copy_(torch.randn((M, K), generator=gen).to(torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = linear_int8(x, wq, ws, out_dtype=torch.float32)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), rep
    q, s = int8.quantize(x.double().cpu().numpy())
    exact = int8.product(q, s, wq.cpu().numpy()[:, :K], ws.cpu().numpy())
    assert np.all(np.abs(got.cpu().numpy() - exact) <= 2.0 ** -21 * np.abs(exact))


def test_int8_one_token_in_a_graph():
    dev = need_gpu()
    D, I, E, k = 512, 256, 16, 4
    say("int8 one token graph")
    w, x, idx, gate = random_layer(dev, 1, D, I, E, k, 8)
    m, eager = (MoELayer(shape_for(1, D, I, E, k, precision="int8", shared_precision="int8"), device=dev)
                for _ in range(2))
    m.forward(w, x, x, gate, m.schedule(idx))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = m.forward(w, x, x, gate, m.schedule(idx))[1]
    for rep in range(3):
        x.copy_(torch.randn((1, D), device=dev).to(torch.bfloat16))
        idx.copy_(torch.randperm(E, device=dev)[:k].view(1, k))
        want = eager.forward(w, x, x, gate, eager.schedule(idx))[1]
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), rep
    assert m.device_error() == 0


def test_int8_expert_parallel_share():
    # R source ranks: this rank's routed rows equal those of the one-GPU layer on the same tokens
    dev = need_gpu()
    w = synth.Workload("ep", T=96, D=256, I=128, E=8, k=2, I_shared=128, seed=14, routing="gaussian")
    R, L = 2, 4
    say("int8 ep", w)
    inp = synth.make_inputs(w)
    wd = quantised(inp, dev)
    x = inp["x"].to(dev)
    half = w.T // R
    one = make(w, dev)
    res = one(x, None, wd, logits=inp["logits"].to(dev))
    y = one.routed_rows().clone().view(w.T, w.k, w.D)
    A = res["idx"].view(R, half * w.k)
    for rank in range(R):
        for b, C in ((None, None), (40, 80)):
            m = MoELayer(shape_for(half, w.D, w.I, w.E, w.k, I_shared=w.I_shared, R=R, rank=rank,
                                   max_rows=w.T * w.k, minibatch_rows=b, ring_rows=C,
                                   precision="int8", shared_precision="int8"), device=dev)
            sched = m.schedule(A.contiguous())
            mine = {n: (v[rank * L:(rank + 1) * L].contiguous() if n.startswith(("q_", "s_")) else v)
                    for n, v in wd.items()}
            m.routed_rows().fill_(-3.0)  # rows behind the last routed one stay as they were
            m.forward(mine, x, x[rank * half:(rank + 1) * half].contiguous(),
                      res["gate"][rank * half:(rank + 1) * half].contiguous(), sched)
            torch.cuda.synchronize()
            assert m.device_error() == 0
            P = int(sched["offsets"][-1])
            rows = m.routed_rows()
            src = sched["sched"][:P].long()
            assert torch.equal(rows[:P], y.view(-1, w.D)[src]), (rank, b)
            assert (rows[P:] == -3).all()


def test_int8_layer_with_a_scored_router_in_a_graph():
    """Router, schedule and int8 experts as a serving step runs them: captured,
    replayed on new tokens between eager work, each replay equal to the eager step."""
    dev = need_gpu()
    w = synth.Workload("serve", T=12, D=512, I=256, E=32, k=4, I_shared=256, seed=21)
    say("int8 serving step", w)
    inp = synth.make_inputs(w)
    wd = quantised(inp, dev, tiled=True)
    wr = inp["w_router"].to(dev)
    bias = 0.1 * torch.randn(w.E, generator=torch.Generator().manual_seed(1)).to(dev)
    r = router_for(score="sigmoid", groups=8, kept_groups=4, scale=2.5)
    x = inp["x"].to(dev)
    m, eager = make(w, dev, tiled=True), make(w, dev, tiled=True)

    def step(layer):
        return layer(x, wr, wd, router=r, bias=bias)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(m)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(m)
    gen = torch.Generator().manual_seed(3)
    for rep in range(3):
        x.copy_(torch.randn((w.T, w.D), generator=gen).to(torch.bfloat16))
        want = step(eager)
        for n in ("out", "out32", "idx"):
            got[n].zero_()
        g.replay()
        torch.cuda.synchronize()
        for n in ("logits", "idx", "gate", "out", "out32"):
            assert torch.equal(got[n], want[n]), (rep, n)
    assert m.device_error() == 0
    # and the eager step is the oracle's
    want, tol = oracle(w, {**inp, "x": x.cpu()}, got["idx"].cpu().numpy(), got["gate"].cpu().numpy())
    assert np.all(np.abs(got["out32"].cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("T", [2, 40, 400])
def test_int8_layer_keeps_a_bad_token_to_itself(T):
    # a token with an infinity comes out NaN; every other one has the bits it has without it
    dev = need_gpu()
    w = synth.Workload("bad", T=T, D=256, I=128, E=8, k=2, I_shared=128, seed=13, routing="gaussian")
    say("int8 bad token", T)
    inp = synth.make_inputs(w)
    wd = quantised(inp, dev)
    lg, x = inp["logits"].to(dev), inp["x"].to(dev)
    want = make(w, dev)(x, None, wd, logits=lg)["out32"]
    bad = x.clone()
    bad[1, 17] = float("inf")
    got = make(w, dev)(bad, None, wd, logits=lg)["out32"]
    assert torch.isnan(got[1]).all()
    keep = torch.arange(T) != 1
    assert torch.equal(got[keep.to(dev)], want[keep.to(dev)])


def test_int8_wide_experts_with_one_token():
    # wide h rows, of one and two tokens and beside others
    dev = need_gpu()
    for T in (1, 2):
        for I in (20352, 20480, 40704, 41088):
            say("int8 wide", T, I)
            w, x, idx, gate = random_layer(dev, T, 128, I, 2, 1, 9)
            m = MoELayer(shape_for(T, 128, I, 2, 1, precision="int8", shared_precision="int8"), device=dev)
            _, got = m.forward(w, x, x, gate, m.schedule(idx))
            # the same tokens among others take the products that read quantised rows
            pad = 6
            xs = torch.cat([x] + [x[:1]] * pad)
            ids, gs = torch.cat([idx] + [idx[:1]] * pad), torch.cat([gate] + [gate[:1]] * pad)
            m8 = MoELayer(shape_for(T + pad, 128, I, 2, 1, precision="int8", shared_precision="int8"), device=dev)
            _, want = m8.forward(w, xs, xs, gs, m8.schedule(ids))
            torch.cuda.synchronize()
            assert m.device_error() == 0 and torch.equal(got, want[:T])


@pytest.mark.parametrize("T", [1, 2, 5, 40])
def test_int8_layer_with_an_expert_named_twice(T):
    # routes are the caller's: a token may name an expert more than once, and then counts it each time
    dev = need_gpu()
    w = synth.Workload("twice", T=T, D=256, I=128, E=4, k=4, I_shared=128, seed=6, routing="gaussian")
    say("int8 twice", T)
    inp = synth.make_inputs(w)
    idx = torch.zeros((T, 4), dtype=torch.int32)
    idx[:, 2:] = 3
    gate = torch.rand((T, 4), generator=torch.Generator().manual_seed(T))
    m = make(w, dev)
    x = inp["x"].to(dev)
    _, out32 = m.forward(quantised(inp, dev), x, x, gate.to(dev), m.schedule(idx.to(dev)))
    torch.cuda.synchronize()
    assert m.device_error() == 0
    both = torch.stack([gate[:, :2].sum(1), gate[:, 2:].sum(1)], dim=1).numpy()
    want, tol = oracle(w, inp, np.tile(np.array([[0, 3]]), (T, 1)), both)
    assert np.all(np.abs(out32.cpu().numpy() - want) <= tol)


def test_int8_layer_without_tokens():
    dev = need_gpu()
    w = synth.Workload("none", T=4, D=128, I=128, E=4, k=2, I_shared=128, seed=3, routing="gaussian")
    inp = synth.make_inputs(w)
    m = MoELayer(shape_for(0, 128, 128, 4, 2, precision="int8", shared_precision="int8"), device=dev)
    r = m(torch.empty((0, 128), dtype=torch.bfloat16, device=dev), None, quantised(inp, dev),
          logits=torch.empty((0, 4), device=dev))
    assert r["out"].shape == (0, 128) and m.device_error() == 0


@pytest.mark.parametrize("K", [1, 2056])
def test_quantize_more_rows_than_one_launch(K):
    # the rows either side of 2^23 and the last ones, of K = 1 (2^23 + 37 rows) and of rows a workgroup each
    dev = need_gpu()
    rows = (1 << 23) + 37
    say("int8 many rows", rows, K)
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device=dev)
    ids = torch.tensor([0, 1, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, rows - 1], device=dev)
    g = torch.Generator().manual_seed(3)
    x[ids] = torch.randn((6, K), generator=g).to(torch.bfloat16).to(dev)
    q, s = quantize_int8(x)
    want_q, want_s = int8.quantize(x[ids].double().cpu().numpy())
    assert np.array_equal(q[ids][:, :K].cpu().numpy(), want_q)
    assert np.allclose(s[ids].double().cpu().numpy(), want_s, rtol=2.0**-24, atol=0)  # one rounding to fp32
    assert not q[ids][:, K:].any() and int((s != 0).sum()) == 6 and int((q != 0).any(1).sum()) == 6
