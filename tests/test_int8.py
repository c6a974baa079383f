"""8-bit integers on the CPU: the oracle's quantiser against a search over the
integers, and the host-side checks of the entry points."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from mixture_experts_layer_counts_amd import _lib, linear_int8, matmul_int8, quantize_int8, shape_for, tile_int8
from oracle import int8
from tests.test_abi import lib, ws_bytes  # noqa: F401


def test_oracle_quantize_by_search():
    rng = np.random.default_rng(2)
    v = torch.from_numpy(rng.standard_normal((20, 31)).astype(np.float32)).to(torch.bfloat16).double().numpy()
    v[0, :4] = [1.0, 0.5, -0.5, 0.25]
    v[0, 4:] = 0.0
    v[1] = 0.0
    q, s = int8.quantize(v)
    assert np.all(q[1] == 0) and s[1] == 0
    assert q[0, :4].tolist() == [127, 64, -64, 32]  # 63.5 to even, 31.75
    for r in range(20):
        m = max(abs(Fraction(float(x))) for x in v[r])
        for x, got in zip(v[r], q[r]):
            if m == 0:
                continue
            t = Fraction(float(x)) * 127 / m
            dist = {n: abs(t - n) for n in range(-127, 128)}
            least = min(dist.values())
            best = [n for n, d in dist.items() if d == least]
            assert int(got) in best and (len(best) == 1 or int(got) % 2 == 0)


def test_oracle_ffn_is_close_to_the_unquantised_one():
    rng = np.random.default_rng(4)
    D, I = 256, 128
    x = rng.standard_normal((9, D))
    mats = {"gate": rng.standard_normal((I, D)) / 16, "up": rng.standard_normal((I, D)) / 16,
            "down": rng.standard_normal((D, I)) / 11}
    w = {}
    for n, m in mats.items():
        w["q_" + n], w["s_" + n] = int8.quantize(m)
    got, _ = int8.ffn(x, w, "")
    g = x @ mats["gate"].T
    want = (g / (1 + np.exp(-g)) * (x @ mats["up"].T)) @ mats["down"].T
    # each of the six roundings is uniform within half a step m / 127, m about 3.5 standard
    # deviations: 0.8% of a standard deviation each, so near 2% in all
    assert np.sqrt(np.mean((got - want) ** 2) / np.mean(want ** 2)) < 0.04


FAKE, OTHER, ODD = (ctypes.c_void_p(v) for v in (4096, 8192, 8200))  # never dereferenced


def test_int8_shapes(lib):  # noqa: F811
    for D, I, code in ((128, 128, 0), (7168, 2048, 0), (128, 64, -2), (192, 128, -2)):
        assert ws_bytes(lib, shape_for(T=64, D=D, I=I, E=8, k=2, I_shared=64, precision="int8"))[0] == code
        assert ws_bytes(lib, shape_for(T=64, D=D, I=64, E=8, k=2, I_shared=I, shared_precision="int8"))[0] == code
    assert ws_bytes(lib, shape_for(T=64, D=128, I=128, E=8, k=2, precision="int8", pipeline=True))[0] == -2
    n = ctypes.c_size_t(0)
    s = shape_for(T=64, D=128, I=128, E=8, k=2, precision="int8")
    assert lib.moe_backward_workspace_bytes(ctypes.byref(s), ctypes.byref(n)) == -2


@pytest.mark.parametrize("routed,shared", [("int8", "bf16"), ("bf16", "int8")])
def test_int8_forward_needs_scales_and_alignment(lib, routed, shared):  # noqa: F811
    s = shape_for(T=64, D=128, I=128, E=8, k=2, precision=routed, shared_precision=shared)
    _, n = ws_bytes(lib, s)
    w = _lib.MoeWeights()
    names = [f for f, _ in _lib.MoeWeights._fields_]

    def run():
        return lib.moe_forward(ctypes.byref(s), ctypes.byref(w), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE,
                               n, None)
    for f in names:
        if not f.startswith(("s_", "ss_")):
            setattr(w, f, 4096)
    assert run() == -1
    for f in names:
        setattr(w, f, 4096)
    setattr(w, "w_up" if routed == "int8" else "ws_up", 4104)
    assert run() == -1


def test_quantize_int8_refusals(lib):  # noqa: F811
    f = lib.moe_quantize_int8
    assert f(FAKE, 2, 4, 64, OTHER, FAKE, None) == -1   # dtype
    assert f(FAKE, 0, -1, 64, OTHER, FAKE, None) == -1
    assert f(FAKE, 0, 4, 0, OTHER, FAKE, None) == -1
    assert f(None, 0, 4, 64, OTHER, FAKE, None) == -1
    assert f(FAKE, 0, 4, 64, FAKE, FAKE, None) == -1    # in place
    assert f(FAKE, 0, 4, 64, ODD, FAKE, None) == -1     # q not 16-byte aligned
    assert f(ctypes.c_void_p(4098), 1, 4, 64, OTHER, FAKE, None) == -1
    assert f(FAKE, 0, 1 << 31, 64, OTHER, FAKE, None) == -2
    assert f(FAKE, 0, 0, 64, OTHER, FAKE, None) == 0    # nothing to do: no launch


def test_matmul_int8_refusals(lib):  # noqa: F811
    def f(M=4, N=8, K=128, a=FAKE, sa=FAKE, b=FAKE, sb=FAKE, out=OTHER, dt=0):
        return lib.moe_matmul_int8(a, sa, M, b, sb, N, K, out, dt, None)
    assert f(dt=2) == -1 and f(K=0) == -1 and f(K=96) == -1 and f(M=-1) == -1 and f(N=-1) == -1
    for n in ("a", "sa", "b", "sb", "out"):
        assert f(**{n: None}) == -1, n
    for n in ("a", "b", "out"):
        assert f(**{n: ODD}) == -1, n
    assert f(sa=ctypes.c_void_p(4097)) == -1
    assert f(K=65536 + 128) == -2 and f(M=1 << 24) == -2 and f(N=1 << 24) == -2 and f(M=1 << 32) == -2
    assert f(M=0) == 0 and f(N=0) == 0


def test_binding_refusals():
    host = torch.zeros((4, 128))
    q, s = torch.zeros((4, 128), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(TypeError):
        quantize_int8([1.0])
    with pytest.raises(ValueError):
        quantize_int8(host)  # not on a device
    with pytest.raises(ValueError):
        quantize_int8(host.half())
    with pytest.raises(ValueError):
        matmul_int8(q, s, q, s)
    with pytest.raises(TypeError):
        matmul_int8(None, s, q, s)
    with pytest.raises(ValueError):
        linear_int8(host, q, s)
    with pytest.raises(ValueError):
        tile_int8(torch.zeros((1, 4, 128), dtype=torch.uint8))
    with pytest.raises(KeyError):
        shape_for(T=1, D=128, I=128, E=4, k=1, precision="int4")


@pytest.mark.parametrize("precision", ["bf16", "mxfp8", "int8"])
def test_forward_without_tokens_still_checks_its_weights(lib, precision):  # noqa: F811
    s = shape_for(T=0, D=128, I=128, E=8, k=2, precision=precision, shared_precision=precision)
    _, n = ws_bytes(lib, s)
    w = _lib.MoeWeights()
    names = [f for f, _ in _lib.MoeWeights._fields_]
    if precision == "bf16":
        names = [f for f in names if f.startswith("w")]

    def run(weights=ctypes.byref(w), offsets=FAKE):
        return lib.moe_forward(ctypes.byref(s), weights, None, None, None, offsets, None, None, None, None, FAKE, n,
                               None)
    for f in names:
        setattr(w, f, 4096)
    assert run() == 0  # no rows: no pointer to them, no launch
    assert run(weights=None) == -1 and run(offsets=None) == -1
    for f in names:
        setattr(w, f, None)
        assert run() == -1, f
        setattr(w, f, 4096)
    if precision == "int8":
        w.ws_down = 4104
        assert run() == -1
