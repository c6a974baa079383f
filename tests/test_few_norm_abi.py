"""moe_few's and moe_block_norm's answers on the host, before any launch (CPU)."""

import ctypes
import os

import pytest

from mixture_experts_layer_counts_amd import _lib, router_for, shape_for


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_counts_amd import build
        build.build()
    return _lib.load()


def P(v):
    return ctypes.c_void_p(v)


def few(lib, s, router=None, w=None, ws_bytes=1 << 40, **kw):
    a = {n: P(4096 * (i + 1)) for i, n in enumerate(("x", "w_router", "logits", "idx", "gate", "out", "out32", "ws"))}
    a["bias"] = None
    a.update(kw)
    if w is None:
        w = _lib.MoeWeights(*([4096] * len(_lib.MoeWeights._fields_)))
    return lib.moe_few(ctypes.byref(s), ctypes.byref(w), None if router is None else ctypes.byref(router), a["x"],
                       a["w_router"], a["bias"], a["logits"], a["idx"], a["gate"], a["out"], a["out32"], a["ws"],
                       ws_bytes, None)


def test_few_refuses(lib):
    s = shape_for(T=4, D=128, I=64, E=8, k=2)
    for kw in (dict(x=None), dict(x=P(4104)), dict(w_router=P(4100)), dict(logits=None), dict(idx=None),
               dict(gate=P(4098)), dict(out=None), dict(out=P(4100)), dict(out32=P(4104)), dict(ws=None),
               dict(ws=P(4112)), dict(bias=P(4096)), dict(w=_lib.MoeWeights())):
        assert few(lib, s, **kw) == -1, kw
    assert few(lib, s, ws_bytes=64) == -3
    bad = router_for(groups=3)
    assert few(lib, s, router=bad) == -1
    # other shapes: too many tokens, 8-bit integers, several ranks
    assert few(lib, shape_for(T=65, D=128, I=64, E=8, k=2)) == -2
    assert few(lib, shape_for(T=4, D=128, I=128, E=8, k=2, precision="int8")) == -2
    assert few(lib, shape_for(T=4, D=128, I=64, E=8, k=2, I_shared=128, shared_precision="int8")) == -2
    assert few(lib, shape_for(T=4, D=128, I=64, E=8, k=2, R=2)) == -2
    # MXFP8 needs its scales
    mx = shape_for(T=4, D=128, I=128, E=8, k=2, I_shared=64, precision="mxfp8")
    w = _lib.MoeWeights(*([4096] * len(_lib.MoeWeights._fields_)))
    w.s_down = None
    assert few(lib, mx, w=w) == -1
    # no tokens: nothing to do, and their pointers may be NULL
    assert few(lib, shape_for(T=0, D=128, I=64, E=8, k=2), x=None, logits=None, idx=None, gate=None, out=None) == 0


def test_few_workspace(lib):
    def size(**kw):
        n = ctypes.c_size_t()
        s = shape_for(**{**dict(T=64, D=2048, I=768, E=128, k=8, minibatch_rows=64, ring_rows=64), **kw})
        assert lib.moe_workspace_bytes(ctypes.byref(s), ctypes.byref(n)) == 0
        return n.value
    # h and the experts' rows in 32 bits, for the shapes it serves
    assert size() > 4 * (512 * 768 + 64 * 768) + 4 * (512 + 64) * 2048
    assert size(T=65) < size()


def norm(**kw):
    n = _lib.MoeNorm()
    n.T, n.D, n.gate_rows, n.scale, n.eps = 16, 64, 0, 1.0, 1e-6
    for k, v in kw.items():
        setattr(n, k, v)
    return n


BIG = 1 << 20


def forward(lib, n, **kw):
    a = dict(x=P(BIG), y=P(2 * BIG), post=P(3 * BIG), gate=None, pre=P(4 * BIG), rng=None, z=P(5 * BIG), h=P(6 * BIG))
    a.update(kw)
    return lib.moe_block_norm(ctypes.byref(n), *[a[k] for k in ("x", "y", "post", "gate", "pre", "rng", "z", "h")], None)


def backward(lib, n, nbytes=None, **kw):
    a = dict(z=P(BIG), y=P(2 * BIG), dz=P(3 * BIG), dh=P(4 * BIG), post=P(5 * BIG), gate=None, pre=P(6 * BIG), rng=None,
             dx=P(7 * BIG), dy=P(8 * BIG), dpost=P(9 * BIG), dgate=None, dpre=P(10 * BIG), ws=P(11 * BIG))
    a.update(kw)
    need = ctypes.c_size_t(0)
    lib.moe_block_norm_backward_workspace_bytes(ctypes.byref(n), ctypes.byref(need))
    return lib.moe_block_norm_backward(
        ctypes.byref(n), *[a[k] for k in ("z", "y", "dz", "dh", "post", "gate", "pre", "rng", "dx", "dy", "dpost", "dgate",
                                          "dpre", "ws")], need.value if nbytes is None else nbytes, None)


@pytest.mark.parametrize("field,value,code", [
    ("T", -1, -1), ("T", 1 << 31, -1), ("D", 0, -1), ("D", 7, -2), ("D", 16385, -2), ("gate_rows", 3, -1),
    ("gate_rows", -1, -1), ("x_dtype", 2, -1), ("y_dtype", -1, -1), ("w_dtype", 5, -1), ("dh_dtype", 2, -1),
    ("scale", float("nan"), -1), ("eps", -1.0, -1), ("eps", float("inf"), -1), ("weight_offset", float("inf"), -1),
    ("dropout", 1.0, -1), ("dropout", -0.5, -1), ("dropout", float("nan"), -1),
])
def test_norm_sizes(lib, field, value, code):
    n = norm(**{field: value})
    assert forward(lib, n) == code
    assert backward(lib, n) == code
    assert lib.moe_block_norm_backward_workspace_bytes(ctypes.byref(n), ctypes.byref(ctypes.c_size_t())) == code


def test_norm_arguments(lib):
    n = norm()
    for kw in (dict(x=None), dict(z=None), dict(h=None), dict(pre=None), dict(y=None), dict(gate=P(7 * BIG)),
               dict(rng=P(7 * BIG)), dict(x=P(BIG + 1)), dict(z=P(BIG)), dict(h=P(2 * BIG + 2)), dict(h=P(5 * BIG + 16)),
               dict(z=P(4 * BIG)), dict(y=None, post=None, pre=None, h=None)):
        assert forward(lib, n, **kw) == -1, kw
    for kw in (dict(dx=None), dict(dy=None), dict(dh=None), dict(dpost=None), dict(dpre=None), dict(z=None),
               dict(dgate=P(12 * BIG)), dict(dx=P(3 * BIG)), dict(dy=P(2 * BIG)), dict(ws=P(7 * BIG)), dict(ws=None),
               dict(dx=P(8 * BIG)), dict(dpre=P(10 * BIG + 2))):
        assert backward(lib, n, **kw) == -1, kw
    assert backward(lib, n, nbytes=3) == -3
    # a gate, and dropout, with what they need
    assert forward(lib, norm(gate_rows=4)) == -1
    assert forward(lib, norm(dropout=0.1)) == -1
    # no rows
    assert forward(lib, norm(T=0), x=None, y=None, z=None, h=None) == 0


def test_norm_numbers_beyond_fp32(lib):
    for kw in (dict(scale=1e39), dict(scale=3e38, dropout=0.5), dict(eps=1e39), dict(weight_offset=-1e39)):
        assert forward(lib, norm(**kw), rng=P(7 * BIG) if "dropout" in kw else None) == -1, kw
