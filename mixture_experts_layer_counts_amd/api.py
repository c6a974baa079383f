"""Thin torch binding of libmoe.so: argument checks and marshalling only.

Torch supplies device memory and the current HIP stream; the C calls do all
of the work.  Names follow include/moe.h: ``route``, ``schedule``,
``forward``, ``quantize_mxfp8``, ``pack_mxfp8_scales``, ``quantize_int8``,
``matmul_int8``, ``linear_int8``, ``few`` and ``block_norm``.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import Dict, Optional, Tuple

import torch

from . import _lib


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    """The current device's current stream, as a handle (the handle alone: a
    torch.cuda.Stream object would cost as much as a kernel launch)."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


_HERE = contextlib.nullcontext()


def _on(device: torch.device):
    """``device`` as the current one (nothing to do where it already is)."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _need(t: torch.Tensor, name: str, dtype, shape, device: torch.device) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def shape_for(T: int, D: int, I: int, E: int, k: int, I_shared: Optional[int] = None,
              minibatch_rows: Optional[int] = None, ring_rows: Optional[int] = None,
              precision: str = "bf16", R: int = 1, rank: int = 0, max_rows: Optional[int] = None,
              shared_precision: str = "bf16", pipeline: bool = False, mem_workgroups: int = 0,
              weights_tiled: bool = False) -> _lib.MoeShape:
    """A moe_shape for one GPU (R = 1) or for rank ``rank`` of R source ranks.
    ``precision`` is that of the routed experts, ``shared_precision`` that of
    the shared expert (bf16 unless MXFP8 or int8 is asked for).  ``pipeline`` runs the
    routed minibatch loop as one persistent kernel, ``mem_workgroups`` of
    whose workgroups gather the minibatches the ring does not hold at once.
    ``weights_tiled``: the routed weights come K-tiled (``tile_bf16``,
    ``tile_mxfp8``, ``tile_int8``)."""
    L = E // R
    max_rows = T * k if max_rows is None else max_rows
    b = minibatch_rows or max(max_rows, 1)
    C = ring_rows or b
    s = _lib.MoeShape()
    s.T, s.D, s.I, s.I_shared, s.E_total, s.k = T, D, I, I if I_shared is None else I_shared, E, k
    s.num_src_ranks, s.rank, s.experts_per_rank, s.tokens_per_src_rank = R, rank, L, T
    s.max_rows, s.minibatch_rows, s.ring_rows = max_rows, b, C
    s.precision = _lib.PRECISIONS[precision]
    s.shared_precision = _lib.PRECISIONS[shared_precision]
    s.pipeline, s.mem_workgroups = int(bool(pipeline)), mem_workgroups
    s.weights_tiled = int(bool(weights_tiled))
    return s


def router_for(score: str = "sigmoid", groups: int = 1, kept_groups: int = 1, group_score: str = "top2",
               renorm: bool = True, scale: float = 1.0) -> _lib.MoeRouter:
    """A moe_router: how ``route`` scores and chooses experts (moe_route_scored).
    ``score`` is "sigmoid" or "softmax"; of ``groups`` groups of consecutive
    experts the ``kept_groups`` best stay, ranked by their largest value
    (``group_score`` "max") or the sum of their two largest ("top2");
    ``renorm`` divides the gates by their sum, ``scale`` multiplies them."""
    if score not in _lib.SCORES:
        raise ValueError(f"score must be one of {sorted(_lib.SCORES)}, got {score!r}")
    if group_score not in _lib.GROUP_SCORES:
        raise ValueError(f"group_score must be one of {sorted(_lib.GROUP_SCORES)}, got {group_score!r}")
    r = _lib.MoeRouter()
    r.score, r.groups, r.kept_groups = _lib.SCORES[score], groups, kept_groups
    r.group_score, r.renorm, r.scale = _lib.GROUP_SCORES[group_score], int(bool(renorm)), scale
    return r


def _weight_specs(s: _lib.MoeShape):
    """(moe_weights field, name in ``weights``, dtype, shape) of every tensor ``forward`` reads."""
    L, D, I, Is = s.experts_per_rank, s.D, s.I, s.I_shared
    routed = (("gate", I, D), ("up", I, D), ("down", D, I))
    shared = (("gate", Is, D), ("up", Is, D), ("down", D, Is))
    out = []
    for n, N, K in routed:
        if s.precision == _lib.MOE_BF16:
            # row-major [L, N, K], or K-tiled [L, K/64, N, 64] (tile_bf16)
            out.append(("w_" + n, "w_" + n, torch.bfloat16, (L, K // 64, N, 64) if s.weights_tiled else (L, N, K)))
            continue
        # row-major [L, N, K] bytes, or K-tiled [L, K/128, N, 128] (tile_mxfp8, tile_int8)
        shp = (L, K // 128, N, 128) if s.weights_tiled else (L, N, K)
        if s.precision == _lib.MOE_INT8:  # int8 and a scale per row (quantize_int8)
            out += [("w_" + n, "q_" + n, torch.int8, shp), ("s_" + n, "s_" + n, torch.float32, (L, N))]
        else:
            out += [("w_" + n, "q_" + n, torch.uint8, shp), ("s_" + n, "s_" + n, torch.uint8, (L, K // 128, N, 4))]
    for n, N, K in shared:
        if s.shared_precision == _lib.MOE_BF16:
            out.append(("ws_" + n, "ws_" + n, torch.bfloat16, (N, K)))
        elif s.shared_precision == _lib.MOE_INT8:
            out += [("ws_" + n, "qs_" + n, torch.int8, (N, K)), ("ss_" + n, "ss_" + n, torch.float32, (N,))]
        else:  # E4M3 bytes and packed scales (quantize_mxfp8, pack_mxfp8_scales)
            out += [("ws_" + n, "qs_" + n, torch.uint8, (N, K)), ("ss_" + n, "ss_" + n, torch.uint8, (K // 128, N, 4))]
    return out


class MoELayer:
    """One layer's shape plus its device workspace, on ``device``."""

    def __init__(self, shape: _lib.MoeShape, device="cuda"):
        self.lib = _lib.load()
        self.shape = shape
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        nbytes = ctypes.c_size_t(0)
        _lib.check("moe_workspace_bytes", self.lib.moe_workspace_bytes(ctypes.byref(shape), ctypes.byref(nbytes)))
        self.ws_bytes = nbytes.value
        # the caching allocator hands out 512-byte aligned blocks
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=self.device)
        with _on(self.device):
            _lib.check("moe_workspace_init",
                       self.lib.moe_workspace_init(ctypes.byref(shape), _ptr(self.ws), self.ws_bytes, _stream()))
        self._weight_specs = _weight_specs(shape)

    # -- sizes -------------------------------------------------------------
    @property
    def T(self):
        return self.shape.T

    @property
    def k(self):
        return self.shape.k

    # -- moe_route ---------------------------------------------------------
    def route(self, x: Optional[torch.Tensor], w_router: Optional[torch.Tensor],
              logits: Optional[torch.Tensor] = None, router: Optional[_lib.MoeRouter] = None,
              bias: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(logits, idx, gate).  Without ``router``: top-k of the logits with
        renormalised softmax gates (moe_route).  With one (``router_for``):
        moe_route_scored, with ``bias`` [E] fp32 added to the scores for the
        choice alone."""
        s, dev = self.shape, self.device
        if bias is not None:
            if router is None:
                raise ValueError("a bias needs a router")
            _need(bias, "bias", torch.float32, (s.E_total,), dev)
        if x is None:
            if logits is None:
                raise ValueError("given-logits mode needs logits")
            _need(logits, "logits", torch.float32, (s.T, s.E_total), dev)
        else:
            _need(x, "x", torch.bfloat16, (s.T, s.D), dev)
            _need(w_router, "w_router", torch.bfloat16, (s.E_total, s.D), dev)
            logits = torch.empty((s.T, s.E_total), dtype=torch.float32, device=dev)
        idx = torch.empty((s.T, s.k), dtype=torch.int32, device=dev)
        gate = torch.empty((s.T, s.k), dtype=torch.float32, device=dev)
        with _on(dev):
            if router is None:
                _lib.check("moe_route", self.lib.moe_route(ctypes.byref(s), _ptr(x), _ptr(w_router), _ptr(logits),
                                                           _ptr(idx), _ptr(gate), _ptr(self.ws), self.ws_bytes,
                                                           _stream()))
            else:
                _lib.check("moe_route_scored", self.lib.moe_route_scored(
                    ctypes.byref(s), ctypes.byref(router), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(logits),
                    _ptr(idx), _ptr(gate), _ptr(self.ws), self.ws_bytes, _stream()))
        return logits, idx, gate

    def route_backward(self, logits: torch.Tensor, idx: torch.Tensor, dgate: torch.Tensor,
                       router: _lib.MoeRouter) -> torch.Tensor:
        """The gradient [T, E] fp32 of the logits for a gradient ``dgate`` of
        the gates that ``route`` returned with ``router`` (moe_route_backward)."""
        s, dev = self.shape, self.device
        _need(logits, "logits", torch.float32, (s.T, s.E_total), dev)
        _need(idx, "idx", torch.int32, (s.T, s.k), dev)
        _need(dgate, "dgate", torch.float32, (s.T, s.k), dev)
        dlogits = torch.empty((s.T, s.E_total), dtype=torch.float32, device=dev)
        with _on(dev):
            _lib.check("moe_route_backward", self.lib.moe_route_backward(
                ctypes.byref(s), ctypes.byref(router), _ptr(logits), _ptr(idx), _ptr(dgate), _ptr(dlogits),
                _ptr(self.ws), self.ws_bytes, _stream()))
        return dlogits

    # -- moe_schedule ------------------------------------------------------
    def schedule(self, routes: torch.Tensor) -> Dict[str, torch.Tensor]:
        s, dev = self.shape, self.device
        NK = s.T * s.k
        routes = routes.reshape(s.num_src_ranks, NK)
        _need(routes, "routes", torch.int32, (s.num_src_ranks, NK), dev)
        L = s.experts_per_rank
        out = {
            "counts": torch.empty(L, dtype=torch.int32, device=dev),
            "offsets": torch.empty(L + 1, dtype=torch.int32, device=dev),
            "sched": torch.empty((max(s.max_rows, 1),), dtype=torch.int32, device=dev),
            "route_dst": torch.empty(s.num_src_ranks * NK, dtype=torch.int32, device=dev),
        }
        with _on(dev):
            _lib.check("moe_schedule", self.lib.moe_schedule(
                ctypes.byref(s), _ptr(routes), _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["sched"]),
                _ptr(out["route_dst"]), _ptr(self.ws), self.ws_bytes, _stream()))
        return out

    def _weights(self, weights: Dict[str, torch.Tensor]) -> _lib.MoeWeights:
        w = _lib.MoeWeights()
        for field, name, dtype, shp in self._weight_specs:
            t = weights[name]
            _need(t, name, dtype, shp, self.device)
            setattr(w, field, t.data_ptr())
        return w

    # -- moe_forward -------------------------------------------------------
    def forward(self, weights: Dict[str, torch.Tensor], x_src: torch.Tensor, x_local: torch.Tensor,
                gate: torch.Tensor, sched: Dict[str, torch.Tensor], out32: bool = True,
                out: Optional[torch.Tensor] = None, out_f32: Optional[torch.Tensor] = None):
        s, dev, D = self.shape, self.device, self.shape.D
        _need(x_local, "x_local", torch.bfloat16, (s.T, D), dev)
        _need(x_src, "x_src", torch.bfloat16, (s.num_src_ranks * s.T, D), dev)
        _need(gate, "gate", torch.float32, (s.T, s.k), dev)
        w = self._weights(weights)
        if out is None:
            out = torch.empty((s.T, D), dtype=torch.bfloat16, device=dev)
        _need(out, "out", torch.bfloat16, (s.T, D), dev)
        if out32 and out_f32 is None:
            out_f32 = torch.empty((s.T, D), dtype=torch.float32, device=dev)
        if out_f32 is not None:
            _need(out_f32, "out32", torch.float32, (s.T, D), dev)
        with _on(dev):
            _lib.check("moe_forward", self.lib.moe_forward(
                ctypes.byref(s), ctypes.byref(w), _ptr(x_src), _ptr(x_local), _ptr(gate), _ptr(sched["offsets"]),
                _ptr(sched["sched"]), _ptr(sched["route_dst"]), _ptr(out), _ptr(out_f32), _ptr(self.ws),
                self.ws_bytes, _stream()))
        return out, out_f32

    # -- moe_few -----------------------------------------------------------
    def few(self, x: torch.Tensor, w_router: Optional[torch.Tensor], weights: Dict[str, torch.Tensor],
            logits: Optional[torch.Tensor] = None, router: Optional[_lib.MoeRouter] = None,
            bias: Optional[torch.Tensor] = None, out32: bool = True) -> Dict[str, Optional[torch.Tensor]]:
        """The whole layer for at most 64 tokens in one launch (moe_few), from x
        or from given ``logits``: logits, idx, gate, out and out32 (None unless
        asked for).  bf16 and MXFP8 experts, one GPU."""
        s, dev = self.shape, self.device
        T, D, E, k = s.T, s.D, s.E_total, s.k
        _need(x, "x", torch.bfloat16, (T, D), dev)
        if bias is not None:
            if router is None:
                raise ValueError("a bias needs a router")
            _need(bias, "bias", torch.float32, (E,), dev)
        if logits is not None:
            _need(logits, "logits", torch.float32, (T, E), dev)
            w_router = None
        else:
            _need(w_router, "w_router", torch.bfloat16, (E, D), dev)
        w = self._weights(weights)
        with _on(dev):
            if logits is None:
                logits = torch.empty((T, E), dtype=torch.float32, device=dev)
            idx = torch.empty((T, k), dtype=torch.int32, device=dev)
            gate = torch.empty((T, k), dtype=torch.float32, device=dev)
            out = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
            out_f32 = torch.empty((T, D), dtype=torch.float32, device=dev) if out32 else None
            _lib.check("moe_few", self.lib.moe_few(
                ctypes.byref(s), ctypes.byref(w), None if router is None else ctypes.byref(router), _ptr(x),
                _ptr(w_router), _ptr(bias), _ptr(logits), _ptr(idx), _ptr(gate), _ptr(out), _ptr(out_f32),
                _ptr(self.ws), self.ws_bytes, _stream()))
        return {"logits": logits, "idx": idx, "gate": gate, "out": out, "out32": out_f32}

    # -- whole layer -------------------------------------------------------
    def __call__(self, x: torch.Tensor, w_router: Optional[torch.Tensor], weights: Dict[str, torch.Tensor],
                 logits: Optional[torch.Tensor] = None, router: Optional[_lib.MoeRouter] = None,
                 bias: Optional[torch.Tensor] = None):
        """route + schedule + forward for R = 1 (from x, or from given logits)."""
        lg, idx, gate = self.route(None if logits is not None else x, w_router, logits, router, bias)
        sched = self.schedule(idx)
        out, out32 = self.forward(weights, x, x, gate, sched)
        return {"logits": lg, "idx": idx, "gate": gate, "out": out, "out32": out32, **sched}

    def block(self, x: torch.Tensor, w_router: Optional[torch.Tensor], weights: Dict[str, torch.Tensor],
              pre_weight: torch.Tensor, post_weight: Optional[torch.Tensor] = None,
              gate: Optional[torch.Tensor] = None, next_weight: Optional[torch.Tensor] = None, scale: float = 1.0,
              eps: float = 1e-6, weight_offset: float = 0.0, dropout: float = 0.0,
              rng: Optional[torch.Tensor] = None, router: Optional[_lib.MoeRouter] = None,
              bias: Optional[torch.Tensor] = None, train: bool = False) -> Dict[str, Optional[torch.Tensor]]:
        """The layer as a block of a model, for R = 1: h = norm(x) * pre_weight, the
        layer's out of h, and z = x + scale * gate * drop(norm(out) * post_weight) with
        h_next = norm(z) * next_weight for what follows (``block_norm``).  Calls for
        few tokens run the layer in one launch (``few``) unless ``train`` is set, which
        keeps what ``MoEBackward.block`` needs.  The layer's results, h, z and h_next."""
        s = self.shape
        _, h = block_norm(x, pre_weight=pre_weight, eps=eps, weight_offset=weight_offset)
        quantised = _lib.MOE_INT8 in (s.precision, s.shared_precision)
        # few against the layer's own launches, captured, us: 7168 x 2048 of 256 experts 1 token 193 and 364, 16
        # 1545 and 1683, 64 3349 and 3314; 2048 x 768 of 128 68 and 122, 217 and 246, 291 and 307 (MXFP8 69 and 97,
        # 194 and 193, 221 and 225); 4096 x 14336 of 8 232 and 508, 574 and 708, 749 and 710; 256 x 128 of 8 29 and
        # 44, 35 and 45, 39 and 46.  So few for all that it serves: where it is slower, at 64 tokens, it is by 1 to 7 %.
        if train or s.T > _lib.FEW_TOKENS or s.num_src_ranks != 1 or quantised:
            r = self(h, w_router, weights, router=router, bias=bias)
        else:
            r = self.few(h, w_router, weights, router=router, bias=bias, out32=False)
        z, h_next = block_norm(x, r["out"], post_weight=post_weight, gate=gate, pre_weight=next_weight, scale=scale,
                               eps=eps, weight_offset=weight_offset, dropout=dropout, rng=rng)
        return {**r, "h": h, "z": z, "h_next": h_next}

    def routed_rows(self) -> torch.Tensor:
        """The routed output rows moe_forward left in the workspace (a view,
        bf16 [n, D]): by route t*k+s when R == 1, by schedule position when R > 1."""
        addr, n = ctypes.c_void_p(), ctypes.c_int64()
        _lib.check("moe_routed_rows", self.lib.moe_routed_rows(ctypes.byref(self.shape), _ptr(self.ws), self.ws_bytes,
                                                               ctypes.byref(addr), ctypes.byref(n)))
        off, D = addr.value - self.ws.data_ptr(), self.shape.D
        return self.ws[off:off + n.value * D * 2].view(torch.bfloat16).view(n.value, D)

    def device_error(self) -> int:
        code = ctypes.c_int32(0)
        with _on(self.device):
            _lib.check("moe_get_device_error", self.lib.moe_get_device_error(
                ctypes.byref(self.shape), _ptr(self.ws), self.ws_bytes, _stream(), ctypes.byref(code)))
        return code.value


def schedule_static(shape: _lib.MoeShape, routes: torch.Tensor, dev_error: torch.Tensor) -> Dict[str, torch.Tensor]:
    """moe_schedule_static: the schedule of ``routes`` [R, N*k] int32 with no
    workspace (the library's fixed scratch array); device error bits are
    OR-ed into ``dev_error`` (one int32 on the same device)."""
    lib = _lib.load()
    dev = routes.device
    NK = shape.T * shape.k
    routes = routes.reshape(shape.num_src_ranks, NK)
    _need(routes, "routes", torch.int32, (shape.num_src_ranks, NK), dev)
    _need(dev_error, "dev_error", torch.int32, (1,), dev)
    L = shape.experts_per_rank
    out = {
        "counts": torch.empty(L, dtype=torch.int32, device=dev),
        "offsets": torch.empty(L + 1, dtype=torch.int32, device=dev),
        "sched": torch.empty((max(shape.max_rows, 1),), dtype=torch.int32, device=dev),
        "route_dst": torch.empty(shape.num_src_ranks * NK, dtype=torch.int32, device=dev),
    }
    with _on(dev):
        _lib.check("moe_schedule_static", lib.moe_schedule_static(
            ctypes.byref(shape), _ptr(routes), _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["sched"]),
            _ptr(out["route_dst"]), _ptr(dev_error), _stream()))
    return out


def _weights_struct(shape: _lib.MoeShape, weights: Dict[str, torch.Tensor], dev) -> _lib.MoeWeights:
    L, D, I, Is = shape.experts_per_rank, shape.D, shape.I, shape.I_shared
    w = _lib.MoeWeights()
    for n, shp in (("w_gate", (L, I, D)), ("w_up", (L, I, D)), ("w_down", (L, D, I)), ("ws_gate", (Is, D)),
                   ("ws_up", (Is, D)), ("ws_down", (D, Is))):
        _need(weights[n], n, torch.bfloat16, shp, dev)
        setattr(w, n, _ptr(weights[n]))
    return w


def prepare_backward(shape: _lib.MoeShape, weights: Dict[str, torch.Tensor], w_router: torch.Tensor
                     ) -> Dict[str, torch.Tensor]:
    """The weights rearranged for moe_backward (moe_backward_prepare), once per
    weight set: w_gu, w_gu_t, w_down_t, ws_gu, ws_gu_t, ws_down_t, w_router_t."""
    lib = _lib.load()
    dev = w_router.device
    L, D, I, Is, E = shape.experts_per_rank, shape.D, shape.I, shape.I_shared, shape.E_total
    Ep = (E + 63) // 64 * 64
    w = _weights_struct(shape, weights, dev)
    _need(w_router, "w_router", torch.bfloat16, (E, D), dev)
    out = {"w_gu": (L, 2 * I, D), "w_gu_t": (L, D, 2 * I), "w_down_t": (L, I, D), "ws_gu": (2 * Is, D),
           "ws_gu_t": (D, 2 * Is), "ws_down_t": (Is, D), "w_router_t": (D, Ep)}
    out = {n: torch.empty(shp, dtype=torch.bfloat16, device=dev) for n, shp in out.items()}
    bw = _lib.MoeBwdWeights(*[_ptr(out[n]) for n, _ in _lib.MoeBwdWeights._fields_])
    with _on(dev):
        _lib.check("moe_backward_prepare", lib.moe_backward_prepare(
            ctypes.byref(shape), ctypes.byref(w), _ptr(w_router), ctypes.byref(bw), _stream()))
    return out


class MoEBackward:
    """The workspace of moe_backward for one layer shape, on ``device``."""

    def __init__(self, shape: _lib.MoeShape, device="cuda"):
        self.lib = _lib.load()
        self.shape = shape
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        nbytes = ctypes.c_size_t(0)
        _lib.check("moe_backward_workspace_bytes",
                   self.lib.moe_backward_workspace_bytes(ctypes.byref(shape), ctypes.byref(nbytes)))
        self.ws_bytes = nbytes.value
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=self.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)

    def __call__(self, bw: Dict[str, torch.Tensor], x: torch.Tensor, idx: torch.Tensor, gate: torch.Tensor,
                 sched: Dict[str, torch.Tensor], y_routes: torch.Tensor, dout: torch.Tensor,
                 grads: Optional[Dict[str, torch.Tensor]] = None, router: Optional[_lib.MoeRouter] = None,
                 logits: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
        """The gradients of one forward.  ``router`` and ``logits``: those of
        its ``route`` call, when that had a router (moe_backward_scored)."""
        s, dev = self.shape, self.device
        if (router is None) != (logits is None):
            raise ValueError("router and logits come together")
        if logits is not None:
            _need(logits, "logits", torch.float32, (s.T, s.E_total), dev)
        T, D, I, Is, E, k, L = s.T, s.D, s.I, s.I_shared, s.E_total, s.k, s.experts_per_rank
        _need(x, "x", torch.bfloat16, (T, D), dev)
        _need(dout, "dout", torch.bfloat16, (T, D), dev)
        _need(idx, "idx", torch.int32, (T, k), dev)
        _need(gate, "gate", torch.float32, (T, k), dev)
        _need(y_routes, "y_routes", torch.bfloat16, (T * k, D), dev)
        shapes = {"dx": ((T, D), torch.float32), "dw_gate": ((L, I, D), torch.bfloat16),
                  "dw_up": ((L, I, D), torch.bfloat16), "dw_down": ((L, D, I), torch.bfloat16),
                  "dws_gate": ((Is, D), torch.bfloat16), "dws_up": ((Is, D), torch.bfloat16),
                  "dws_down": ((D, Is), torch.bfloat16), "dw_router": ((E, D), torch.float32)}
        if grads is None:
            grads = {n: torch.empty(shp, dtype=dt, device=dev) for n, (shp, dt) in shapes.items()}
        for n, (shp, dt) in shapes.items():
            _need(grads[n], n, dt, shp, dev)
        g = _lib.MoeGrads(*[_ptr(grads[n]) for n, _ in _lib.MoeGrads._fields_])
        b = _lib.MoeBwdWeights(*[_ptr(bw[n]) for n, _ in _lib.MoeBwdWeights._fields_])
        with _on(dev):
            rest = (_ptr(idx), _ptr(gate), _ptr(sched["offsets"]), _ptr(sched["sched"]), _ptr(sched["route_dst"]),
                    _ptr(y_routes), _ptr(dout), ctypes.byref(g), _ptr(self.err), _ptr(self.ws), self.ws_bytes,
                    _stream())
            if router is None:
                _lib.check("moe_backward", self.lib.moe_backward(ctypes.byref(s), ctypes.byref(b), _ptr(x), *rest))
            else:
                _lib.check("moe_backward_scored", self.lib.moe_backward_scored(
                    ctypes.byref(s), ctypes.byref(router), ctypes.byref(b), _ptr(x), _ptr(logits), *rest))
        return grads

    def block(self, bw: Dict[str, torch.Tensor], x: torch.Tensor, r: Dict[str, torch.Tensor],
              y_routes: torch.Tensor, dz: Optional[torch.Tensor], dh_next: Optional[torch.Tensor],
              pre_weight: torch.Tensor, post_weight: Optional[torch.Tensor] = None,
              gate: Optional[torch.Tensor] = None, next_weight: Optional[torch.Tensor] = None, scale: float = 1.0,
              eps: float = 1e-6, weight_offset: float = 0.0, dropout: float = 0.0,
              rng: Optional[torch.Tensor] = None, router: Optional[_lib.MoeRouter] = None
              ) -> Dict[str, Optional[torch.Tensor]]:
        """The gradients of ``MoELayer.block(..., train=True)``, which returned ``r``,
        for gradients ``dz`` of its z and ``dh_next`` of its h_next: the layer's, with
        dx that of the block's x, and dpre_weight, dpost_weight, dgate, dnext_weight."""
        if any(n not in r for n in ("offsets", "sched", "route_dst")):
            raise ValueError("r has no schedule: it must come from MoELayer.block(..., train=True)")
        opts = dict(eps=eps, weight_offset=weight_offset)
        out = block_norm_backward(r["z"], r["out"], dz, dh_next, post_weight=post_weight, gate=gate,
                                  pre_weight=next_weight, scale=scale, dropout=dropout, rng=rng, **opts)
        grads = self(bw, r["h"], r["idx"], r["gate"], r, y_routes, out["dy"], router=router,
                     logits=None if router is None else r["logits"])
        into = block_norm_backward(x, None, out["dx"], grads["dx"], pre_weight=pre_weight, **opts)
        return {**grads, "dx": into["dx"], "dpre_weight": into["dpre_weight"], "dpost_weight": out["dpost_weight"],
                "dgate": out["dgate"], "dnext_weight": out["dpre_weight"]}

    def device_error(self) -> int:
        torch.cuda.current_stream(self.device).synchronize()
        return int(self.err.item())


def quantize_mxfp8(src: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """MX-quantise a bf16 tensor along its last axis (moe_quantize_mxfp8)."""
    lib = _lib.load()
    if src.dtype != torch.bfloat16 or not src.is_contiguous() or src.device.type != "cuda":
        raise ValueError("src must be a contiguous bf16 device tensor")
    K = src.shape[-1]
    rows = src.numel() // max(K, 1)
    q = torch.empty(src.shape, dtype=torch.uint8, device=src.device)
    sc = torch.empty(src.shape[:-1] + (K // 32,), dtype=torch.uint8, device=src.device)
    with _on(src.device):
        _lib.check("moe_quantize_mxfp8", lib.moe_quantize_mxfp8(_ptr(src), rows, K, _ptr(q), _ptr(sc), _stream()))
    return q, sc


def tile_bf16(w: torch.Tensor) -> torch.Tensor:
    """Row-major bf16 matrices [G, N, K] -> the K-tiled [G, K/64, N, 64]
    that ``forward`` reads with ``weights_tiled`` (moe_tile_bf16)."""
    lib = _lib.load()
    if w.dtype != torch.bfloat16 or not w.is_contiguous() or w.device.type != "cuda" or w.dim() != 3:
        raise ValueError("w must be a contiguous bf16 [G, N, K] device tensor")
    G, N, K = w.shape
    if K % 64:
        raise ValueError("K must be a multiple of 64")
    out = torch.empty((G, K // 64, N, 64), dtype=torch.bfloat16, device=w.device)
    with _on(w.device):
        _lib.check("moe_tile_bf16", lib.moe_tile_bf16(_ptr(w), G, N, K, _ptr(out), _stream()))
    return out


def tile_mxfp8(q: torch.Tensor) -> torch.Tensor:
    """Row-major E4M3 bytes [G, N, K] -> the K-tiled [G, K/128, N, 128] that
    ``forward`` reads with ``weights_tiled`` (moe_tile_bf16 on the bytes taken
    as 2-byte units)."""
    if q.dtype != torch.uint8 or not q.is_contiguous() or q.dim() != 3 or q.shape[2] % 128:
        raise ValueError("q must be contiguous uint8 [G, N, K] with K a multiple of 128")
    G, N, K = q.shape
    return tile_bf16(q.view(torch.bfloat16)).view(torch.uint8).view(G, K // 128, N, 128)


def pack_mxfp8_scales(scale: torch.Tensor) -> torch.Tensor:
    """Row-major MX scales [G, N, K/32] -> the stage-major [G, K/128, N, 4]
    that ``forward`` reads (moe_mxfp8_pack_scales)."""
    lib = _lib.load()
    if scale.dtype != torch.uint8 or not scale.is_contiguous() or scale.device.type != "cuda" or scale.dim() != 3:
        raise ValueError("scale must be a contiguous uint8 [G, N, K/32] device tensor")
    G, N, KS = scale.shape
    if KS % 4:
        raise ValueError("K must be a multiple of 128")
    packed = torch.empty((G, KS // 4, N, 4), dtype=torch.uint8, device=scale.device)
    with _on(scale.device):
        _lib.check("moe_mxfp8_pack_scales", lib.moe_mxfp8_pack_scales(_ptr(scale), G, N, KS * 32, _ptr(packed),
                                                                      _stream()))
    return packed


_INT8_DTYPES = {torch.bfloat16: _lib.DT_BF16, torch.float32: _lib.DT_F32}


def _need_int8_source(t: torch.Tensor, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in _INT8_DTYPES or not t.is_contiguous() or t.device.type != "cuda" or t.dim() < 1:
        raise ValueError(f"{name} must be a contiguous bf16 or fp32 device tensor")
    if t.shape[-1] < 1:
        raise ValueError(f"{name} must have at least one column")


def quantize_int8(src: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows of a bf16 or fp32 tensor [..., K] -> (q [..., Kp] int8, scale [...]
    fp32), Kp = K rounded up to 128 (zeros past K): moe_quantize_int8."""
    lib = _lib.load()
    _need_int8_source(src, "src")
    K = src.shape[-1]
    rows = src.numel() // K
    with _on(src.device):
        q = torch.empty(src.shape[:-1] + ((K + 127) // 128 * 128,), dtype=torch.int8, device=src.device)
        scale = torch.empty(src.shape[:-1], dtype=torch.float32, device=src.device)
        _lib.check("moe_quantize_int8", lib.moe_quantize_int8(_ptr(src), _INT8_DTYPES[src.dtype], rows, K, _ptr(q),
                                                              _ptr(scale), _stream()))
    return q, scale


def matmul_int8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """[M, N] = (a b^T) * a_scale[:, None] * b_scale[None, :] of int8 rows a
    [M, Kp], b [N, Kp] as ``quantize_int8`` returns them (moe_matmul_int8)."""
    lib = _lib.load()
    for t, n in ((a, "a"), (b, "b")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a tensor")
        if t.dim() != 2 or t.device.type != "cuda":
            raise ValueError(f"{n} must be a 2-d device tensor")
    (M, K), dev = a.shape, a.device
    _need(a, "a", torch.int8, (M, K), dev)
    _need(a_scale, "a_scale", torch.float32, (M,), dev)
    _need(b, "b", torch.int8, (b.shape[0], K), dev)
    _need(b_scale, "b_scale", torch.float32, (b.shape[0],), dev)
    if out_dtype not in _INT8_DTYPES:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    with _on(dev):
        out = torch.empty((M, b.shape[0]), dtype=out_dtype, device=dev)
        _lib.check("moe_matmul_int8", lib.moe_matmul_int8(
            _ptr(a), _ptr(a_scale), M, _ptr(b), _ptr(b_scale), b.shape[0], K, _ptr(out), _INT8_DTYPES[out_dtype],
            _stream()))
    return out


@functools.lru_cache(maxsize=4096)
def _linear_ws_bytes(M: int, N: int, K: int) -> int:
    nbytes = ctypes.c_size_t(0)
    _lib.check("moe_linear_int8_workspace_bytes",
               _lib.load().moe_linear_int8_workspace_bytes(M, N, K, ctypes.byref(nbytes)))
    return nbytes.value


def linear_int8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """x [..., K] (bf16 or fp32) -> [..., N]: x's rows quantised (quantize_int8),
    then the product with int8 weights w [N, Kp] and their scales [N], as
    ``quantize_int8`` made them from [N, K].  ``out_dtype``: x's unless given."""
    _need_int8_source(x, "x")
    K = x.shape[-1]
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[1] != (K + 127) // 128 * 128:
        raise ValueError(f"w must be int8 [N, {(K + 127) // 128 * 128}] for {K} columns of x")
    lib, dev = _lib.load(), x.device
    N = w.shape[0]
    _need(w, "w", torch.int8, w.shape, dev)
    _need(w_scale, "w_scale", torch.float32, (N,), dev)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in _INT8_DTYPES:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    M = x.numel() // K
    nbytes = _linear_ws_bytes(M, N, K)
    with _on(dev):
        out = torch.empty(x.shape[:-1] + (N,), dtype=out_dtype, device=dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        _lib.check("moe_linear_int8", lib.moe_linear_int8(
            _ptr(x), _INT8_DTYPES[x.dtype], M, K, _ptr(w), _ptr(w_scale), N, _ptr(out), _INT8_DTYPES[out_dtype],
            _ptr(ws), nbytes, _stream()))
    return out


def tile_int8(q: torch.Tensor) -> torch.Tensor:
    """Row-major int8 matrices [G, N, K] -> the K-tiled [G, K/128, N, 128] that
    ``forward`` reads with ``weights_tiled`` (moe_tile_bf16 on the bytes taken
    as 2-byte units)."""
    if q.dtype != torch.int8:
        raise ValueError("q must be int8")
    return tile_mxfp8(q.view(torch.uint8)).view(torch.int8)


@functools.lru_cache(maxsize=4096)
def _norm_sizes(T, D, gate_rows, x_dtype, y_dtype, w_dtype, dh_dtype, scale, eps, weight_offset, dropout):
    n = _lib.MoeNorm()
    n.T, n.D, n.gate_rows = T, D, gate_rows
    n.x_dtype, n.y_dtype, n.w_dtype, n.dh_dtype = (_INT8_DTYPES[t] for t in (x_dtype, y_dtype, w_dtype, dh_dtype))
    n.scale, n.eps, n.weight_offset, n.dropout = scale, eps, weight_offset, dropout
    return n


def _norm_struct(x: torch.Tensor, y: Optional[torch.Tensor], post_weight, gate, pre_weight, scale: float, eps: float,
                 weight_offset: float, dropout: float, rng, x_name: str, dh=None) -> _lib.MoeNorm:
    """The moe_norm of a call, its inputs checked (not to be changed: calls share it)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{x_name} must be a tensor")
    if x.dim() != 2 or x.dtype not in _INT8_DTYPES or x.device.type != "cuda":
        raise ValueError(f"{x_name} must be a [T, D] bf16 or fp32 device tensor")
    (T, D), dev = x.shape, x.device
    _need(x, x_name, x.dtype, (T, D), dev)
    if y is None and pre_weight is None:
        raise ValueError("y or pre_weight must be given")
    if y is None and (post_weight is not None or gate is not None or dropout):
        raise ValueError("post_weight, gate and dropout need y")
    if y is not None:
        if not isinstance(y, torch.Tensor) or y.dtype not in _INT8_DTYPES:
            raise ValueError("y must be a bf16 or fp32 tensor")
        _need(y, "y", y.dtype, (T, D), dev)
    wtype = None
    for t, n in ((post_weight, "post_weight"), (gate, "gate"), (pre_weight, "pre_weight")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.dtype not in _INT8_DTYPES:
            raise ValueError(f"{n} must be a bf16 or fp32 tensor")
        wtype = wtype or t.dtype
        if n == "gate":
            if t.dim() != 2 or t.shape[0] < 1 or T % t.shape[0]:
                raise ValueError("gate must be [G, D], G a divisor of the rows")
            _need(t, n, wtype, (t.shape[0], D), dev)
        else:
            _need(t, n, wtype, (D,), dev)
    if not 0.0 <= dropout < 1.0 - 2.0 ** -33:  # (its threshold among 32-bit words is below 2^32)
        raise ValueError("dropout must be in [0, 1 - 2^-33)")
    if dropout:
        if rng is None:
            raise ValueError("dropout needs rng")
        _need(rng, "rng", torch.int64, (2,), dev)
    return _norm_sizes(T, D, 0 if gate is None else gate.shape[0], x.dtype, torch.bfloat16 if y is None else y.dtype,
                       torch.bfloat16 if wtype is None else wtype, torch.bfloat16 if dh is None else dh.dtype,
                       float(scale), float(eps), float(weight_offset), float(dropout))


def block_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, *, post_weight: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, pre_weight: Optional[torch.Tensor] = None, scale: float = 1.0,
               eps: float = 1e-6, weight_offset: float = 0.0, dropout: float = 0.0,
               rng: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(z, h) around a layer (moe_block_norm): the residual stream
    z = x + scale * gate * drop(norm(y) * post_weight) behind it, and what the next
    layer reads, h = norm(z) * pre_weight in bf16 (None without pre_weight).
    Without ``y`` z is x itself: the norm before a first layer.  x, y [T, D] bf16 or
    fp32; weights [D] and gate [G, D] (T / G consecutive rows share a row of it) of
    one type; ``weight_offset`` is added to the weights.  ``dropout`` draws its mask
    from ``rng``, int64 [2] on the device (seed and offset), and does not store it."""
    lib = _lib.load()
    n = _norm_struct(x, y, post_weight, gate, pre_weight, scale, eps, weight_offset, dropout, rng, "x")
    dev = x.device
    with _on(dev):
        z = x if y is None else torch.empty_like(x)
        h = None if pre_weight is None else torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
        _lib.check("moe_block_norm", lib.moe_block_norm(
            ctypes.byref(n), _ptr(x), _ptr(y), _ptr(post_weight), _ptr(gate), _ptr(pre_weight),
            _ptr(rng) if dropout else None, None if y is None else _ptr(z), _ptr(h), _stream()))
    return z, h


def block_norm_backward(z: torch.Tensor, y: Optional[torch.Tensor], dz: Optional[torch.Tensor],
                        dh: Optional[torch.Tensor], *, post_weight: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, pre_weight: Optional[torch.Tensor] = None,
                        scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0, dropout: float = 0.0,
                        rng: Optional[torch.Tensor] = None) -> Dict[str, Optional[torch.Tensor]]:
    """The gradients of ``block_norm`` (moe_block_norm_backward) for gradients
    ``dz`` (None: zero) and ``dh`` (with pre_weight) of its results: dx, dy,
    dpost_weight, dgate, dpre_weight, the last three in fp32, each None without its
    input.  ``z``: the stream as block_norm returned it (x, where it had no y); the
    other arguments, ``rng``'s values among them, as in that call."""
    lib = _lib.load()
    if (dh is None) != (pre_weight is None):
        raise ValueError("dh and pre_weight come together")
    if dh is not None and (not isinstance(dh, torch.Tensor) or dh.dtype not in _INT8_DTYPES):
        raise ValueError("dh must be a bf16 or fp32 tensor")
    n = _norm_struct(z, y, post_weight, gate, pre_weight, scale, eps, weight_offset, dropout, rng, "z", dh)
    (T, D), dev = z.shape, z.device
    if dz is not None:
        _need(dz, "dz", z.dtype, (T, D), dev)
    if dh is not None:
        _need(dh, "dh", dh.dtype, (T, D), dev)
    nbytes = ctypes.c_size_t(0)
    _lib.check("moe_block_norm_backward_workspace_bytes",
               lib.moe_block_norm_backward_workspace_bytes(ctypes.byref(n), ctypes.byref(nbytes)))
    with _on(dev):
        def f32(like):
            return None if like is None else torch.empty(like.shape, dtype=torch.float32, device=dev)
        out = {"dx": torch.empty_like(z), "dy": None if y is None else torch.empty_like(y),
               "dpost_weight": f32(post_weight), "dgate": f32(gate), "dpre_weight": f32(pre_weight)}
        ws = torch.empty(max(nbytes.value, 1), dtype=torch.uint8, device=dev)
        _lib.check("moe_block_norm_backward", lib.moe_block_norm_backward(
            ctypes.byref(n), _ptr(z), _ptr(y), _ptr(dz), _ptr(dh), _ptr(post_weight), _ptr(gate), _ptr(pre_weight),
            _ptr(rng) if dropout else None, _ptr(out["dx"]), _ptr(out["dy"]), _ptr(out["dpost_weight"]),
            _ptr(out["dgate"]), _ptr(out["dpre_weight"]), _ptr(ws), nbytes.value, _stream()))
    return out
