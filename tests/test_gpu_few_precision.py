"""How exactly moe_few holds h = SiLU(g) u between its two products, seen through products that are exact.

Every token is a power of two in one column, so g and u are single weights times a power of two, and w_down is the
identity: out32 is what h was kept as (one expert, gate 1, a shared expert of zeros).

* bf16: two terms, both rounded to nearest.  For h in [1, 2) times a power of two the first leaves at most 2^-8 of that
  power, and the second at most half a step of what is left: below 2^-8 its step is 2^-16, so 2^-17.  Before that h
  itself, with u = 2^-24: the exponential's argument is rounded (|g| u of its value, the hardware's 2^x to an ulp), and
  1 + e, its reciprocal and two products round: below (|g| + 6) u of h, twice that of the power.
* MXFP8: h to 2^-19 of its value (32 u: |g| up to 26, beyond which h is below half of the smallest value beside any
  h of g > -10) decides which values of E4M3 it becomes.  Where h / X lies further than 2^-19 of itself from a
  border between two of them there is one answer.  The block's power of two is decided by its largest value the
  same way, so blocks whose largest value lies within 2^-19 of a power of two are left out.
  (Both are products of two 4-bit values where SiLU(g) is all but g, for g above 14: half of those lie at ties of
  the same few bits, or at powers of two.  They are some percent of all.)
"""

import pytest
import torch

from mixture_experts_layer_counts_amd import MoELayer, pack_mxfp8_scales, quantize_mxfp8, shape_for
from tests._gpu import need_gpu, say
from tests.test_gpu_few import mx_round, mx_values

pytestmark = pytest.mark.gpu


def tokens(T, D, g, dev):
    x = torch.zeros((T, D))
    x[torch.arange(T), torch.randperm(D, generator=g)[:T]] = 2.0 ** torch.randint(-1, 2, (T,), generator=g).float()
    return x.to(torch.bfloat16).to(dev)


def silu_mul(x, gate, up):
    a, u = x.double() @ gate.T, x.double() @ up.T
    return a / (1 + torch.exp(-a)) * u


@pytest.mark.parametrize("T,I", [(1, 64), (13, 512), (64, 512)])
def test_bf16_terms(T, I):
    dev = need_gpu()
    say("h in bf16 terms", T, I)
    g = torch.Generator().manual_seed(T)

    def rand(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(dev)
    zero = torch.zeros((64, I), dtype=torch.bfloat16, device=dev)
    w = {"w_gate": rand(1, I, I, std=3.0), "w_up": rand(1, I, I), "ws_gate": zero, "ws_up": zero,
         "w_down": torch.eye(I).to(torch.bfloat16).to(dev)[None].contiguous(), "ws_down": zero.t().contiguous()}
    x = tokens(T, I, g, dev)
    layer = MoELayer(shape_for(T, I, I, 1, 1, I_shared=64), device=dev)
    r = layer.few(x, rand(1, I), w)
    assert bool((r["gate"] == 1).all())
    h = silu_mul(x, w["w_gate"][0].double(), w["w_up"][0].double())
    power = torch.exp2(torch.floor(torch.log2(h.abs().clamp(min=2.0 ** -100))))
    a = (x.double() @ w["w_gate"][0].double().T).abs()
    err = (r["out32"].double() - h).abs() / power
    say("  worst, in 2^-17 of the power of two below h:", float(err.max()) * 2 ** 17)
    assert bool((err <= 2.0 ** -17 + 2 * (a + 6) * 2.0 ** -24).all())


def test_largest_h():
    """An h between bf16's largest value and fp32's stays finite in its two terms."""
    dev = need_gpu()
    eye, zero = torch.eye(64).to(torch.bfloat16), torch.zeros((64, 64), dtype=torch.bfloat16)
    gate, up, down = zero.clone(), zero.clone(), zero.clone()
    gate[0, 0], up[0, 0], down[0, 0] = 1.984375 * 2.0 ** 64, 1.0078125 * 2.0 ** 63, 2.0 ** -100
    w = {"w_gate": gate[None], "w_up": up[None], "w_down": down[None], "ws_gate": zero, "ws_up": zero, "ws_down": zero}
    w = {n: t.contiguous().to(dev) for n, t in w.items()}
    x = eye[:1].contiguous().to(dev)
    r = MoELayer(shape_for(1, 64, 64, 1, 1), device=dev).few(x, zero[:1].contiguous().to(dev), w)
    want = 1.984375 * 1.0078125 * 2.0 ** 27
    assert abs(float(r["out32"][0, 0]) - want) <= 2.0 ** -15 * want


@pytest.mark.parametrize("T,scale", [(16, 12.0), (64, 12.0), (64, 2.0)])
def test_mxfp8_values(T, scale):
    dev = need_gpu()
    N = 2048
    off = 0
    for seed in range(4):
        say("h in MXFP8", T, scale, seed)
        g = torch.Generator().manual_seed(seed)
        dg = torch.Generator(device=dev).manual_seed(seed)

        def mx(v):
            q, s = quantize_mxfp8(v.to(torch.bfloat16))
            return q, pack_mxfp8_scales(s), mx_values(q[0], s[0])
        zero = torch.zeros((64, N), dtype=torch.bfloat16, device=dev)
        w, val = {"ws_gate": zero, "ws_up": zero, "ws_down": zero.t().contiguous()}, {}
        for n, m in (("gate", torch.randn((1, N, N), generator=dg, device=dev) * scale),
                     ("up", torch.randn((1, N, N), generator=dg, device=dev)),
                     ("down", torch.eye(N, device=dev)[None])):
            w["q_" + n], w["s_" + n], val[n] = mx(m)
        assert torch.equal(val["down"], torch.eye(N, device=dev).double())
        x = tokens(T, N, g, dev)
        layer = MoELayer(shape_for(T, N, N, 1, 1, I_shared=64, precision="mxfp8"), device=dev)
        r = layer.few(x, zero[:1].contiguous(), w)
        h = silu_mul(x, val["gate"], val["up"])
        low, high = mx_round(h * (1 - 2.0 ** -19)), mx_round(h * (1 + 2.0 ** -19))
        m = torch.log2(h.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100))
        sure = (low == high) & ((m - m.round()).abs() > 2.0 ** -18).expand(T, N // 32, 32).flatten(-2)
        assert float(sure.double().mean()) > 0.9
        off += int((r["out32"].double() != low)[sure].sum())
    say("  values on the wrong side of a border:", off)
    assert off == 0
