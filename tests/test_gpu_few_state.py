"""moe_few on a workspace that is not fit for it: never initialised, or left by a call that gave up.  Each call says so
in the error word and leaves its outputs as they are, and an initialisation makes the workspace good again.  (The one
wait that gives up here is the kernel's own bounded one, about a second.)"""

import ctypes

import pytest
import torch

from mixture_experts_layer_counts_amd import MoELayer, shape_for
from tests._gpu import need_gpu, say
from tests.test_gpu_few import Case

pytestmark = pytest.mark.gpu

PIPELINE = 0x8
CTL = 256  # the counters' first byte: the draw


def init(layer):
    assert layer.lib.moe_workspace_init(ctypes.byref(layer.shape), ctypes.c_void_p(layer.ws.data_ptr()), layer.ws_bytes,
                                        None) == 0


def clear_error(layer):
    layer.ws[:4].zero_()


class Call:
    """moe_few with outputs of the caller's, filled beforehand."""

    def __init__(self, c):
        self.c = c
        s, dev = c.layer.shape, c.dev
        self.w = c.layer._weights(c.weights)
        self.out = {"logits": torch.empty((s.T, s.E_total), dtype=torch.float32, device=dev),
                    "idx": torch.empty((s.T, s.k), dtype=torch.int32, device=dev),
                    "gate": torch.empty((s.T, s.k), dtype=torch.float32, device=dev),
                    "out": torch.empty((s.T, s.D), dtype=torch.bfloat16, device=dev),
                    "out32": torch.empty((s.T, s.D), dtype=torch.float32, device=dev)}

    def __call__(self):
        for t in self.out.values():
            t.fill_(-7)
        l, c = self.c.layer, self.c
        assert l.lib.moe_few(ctypes.byref(l.shape), ctypes.byref(self.w), None, c.x.data_ptr(), c.w_router.data_ptr(),
                             None, *[self.out[n].data_ptr() for n in ("logits", "idx", "gate", "out", "out32")],
                             l.ws.data_ptr(), l.ws_bytes, None) == 0
        return {n: t.clone() for n, t in self.out.items()}


def untouched(r):
    return all(bool((t == -7).all()) for t in r.values())


@pytest.mark.parametrize("T,prec,byte", [(1, "bf16", 0), (5, "bf16", 0xA5), (40, "mxfp8", 0xFF), (3, "mxfp8", 0x01)])
def test_never_initialised(T, prec, byte):
    dev = need_gpu()
    say("not initialised", T, prec, byte)
    c = Case(dev, T, 256, 128, 12, 3, prec=prec, seed=T)
    call = Call(c)
    want = call()
    assert not untouched(want)
    c.layer.ws.fill_(byte)
    clear_error(c.layer)
    for _ in range(2):
        r = call()
        assert c.layer.device_error() == PIPELINE
        assert untouched(r)
    init(c.layer)
    r = call()
    assert c.layer.device_error() == 0
    assert all(torch.equal(r[n], want[n]) for n in r)


def test_after_a_call_that_gave_up():
    dev = need_gpu()
    c = Case(dev, 6, 128, 64, 8, 2, seed=3)
    call = Call(c)
    want = call()
    say("a draw that begins at 1: item 0 is nobody's, and what waits for it gives up")
    c.layer.ws[CTL:CTL + 4].view(torch.int32).fill_(1)
    call()
    assert c.layer.device_error() == PIPELINE
    clear_error(c.layer)
    r = call()
    assert c.layer.device_error() == PIPELINE  # the counters are not to be trusted
    assert untouched(r)
    # a call of another shape on the same workspace says so too
    other = MoELayer(shape_for(2, 128, 64, 8, 2), device=dev)
    other.ws, other.ws_bytes = c.layer.ws, c.layer.ws_bytes
    clear_error(c.layer)
    other.few(c.x[:2].contiguous(), c.w_router, c.weights)
    assert c.layer.device_error() == PIPELINE
    init(c.layer)
    for _ in range(3):
        r = call()
        assert c.layer.device_error() == 0
        assert all(torch.equal(r[n], want[n]) for n in r)
