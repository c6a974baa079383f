"""Measured operators: scored routing and its gradient, and products in 8-bit
integers (a linear map, and the experts of a mixture-of-experts layer).

``run`` computes one pass of a case's operator, as elementary torch operations
or, with ``own`` set, through this framework's public calls.

Definitions (s: scores, b: bias, l: logits):

* routing: s = sigmoid(l), or softmax(l) over the experts; experts are chosen
  by c = s + b.  With groups, a group of consecutive experts ranks by the sum
  of its two largest c (or by its largest), the best ``kept`` groups stay, and
  the k largest c among their experts are chosen, in falling order, ties to
  the lower index.  Gates are ``scale`` times the chosen s, divided by their
  sum where ``renorm`` is set.  The bias only chooses.
* routing gradient: that of the gates with respect to the logits, the choice
  held fixed, for a given gradient of the gates.
* 8-bit rows: a row v with m = max|v| becomes q = round(127 v / m), ties to
  even, with the scale m / 127 (q = 0 and scale 0 for m = 0).
* linear: y = q(x) w^T with integer products, times the scale of the token
  and of the output channel.
* experts: per token sum_s g_s f_s(x) + f_shared(x), f(x) = W_down q(h),
  h = SiLU(W_gate q(x)) * (W_up q(x)), each product as in linear.
"""

import math

import numpy as np
import torch

own = False

# the sizes of one layer: hidden width, expert width, experts, experts a token
LARGE = {"D": 7168, "I": 2048, "E": 256, "k": 8}
MID = {"D": 2048, "I": 768, "E": 128, "k": 8}


def listed():
    sig = {"score": "sigmoid", "groups": 8, "kept": 4, "top2": True, "bias": True, "renorm": True, "scale": 2.5}
    soft = {"score": "softmax", "groups": 12, "kept": 5, "top2": False, "bias": False, "renorm": False, "scale": 1.0}
    return [
        # one token of a serving step: latency
        {"name": "route_t1", "op": "route", "T": 1, "E": 256, "k": 8, **sig},
        # a training batch or a long prompt at the large layer
        {"name": "route_t8192", "op": "route", "T": 8192, "E": 256, "k": 8, **sig},
        # a ragged batch over more experts, softmax scores, groups of 32 ranked by their best
        {"name": "route_t4099", "op": "route", "T": 4099, "E": 384, "k": 6, **soft},
        # the backward of the two batches above
        {"name": "route_grad_t8192", "op": "route_grad", "T": 8192, "E": 256, "k": 8, **sig},
        {"name": "route_grad_t4099", "op": "route_grad", "T": 4099, "E": 384, "k": 6, **soft},
        # one token through the shared expert's up projection: the weights' stream
        {"name": "linear_m1", "op": "linear", "M": 1, "N": 2048, "K": 7168, "x": "bf16", "y": "bf16"},
        # odd sizes, 32-bit activations
        {"name": "linear_m777", "op": "linear", "M": 777, "N": 1001, "K": 1500, "x": "fp32", "y": "fp32"},
        # a prompt through the shared expert's down projection
        {"name": "linear_m8192", "op": "linear", "M": 8192, "N": 7168, "K": 2048, "x": "bf16", "y": "bf16"},
        # serving: one token, and a batch of 64 that touches most experts
        {"name": "experts_t1", "op": "experts", "T": 1, **LARGE},
        {"name": "experts_t64", "op": "experts", "T": 64, **LARGE},
        # a prompt at the middle layer, and the large layer in full
        {"name": "experts_t4096_mid", "op": "experts", "T": 4096, **MID},
        {"name": "experts_t8192", "op": "experts", "T": 8192, **LARGE},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "linear", "linear", "experts", "experts"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 3, 4, 8, 8, 12, 16])
        size = _log(rng, 2, 384 // groups)
        E = groups * size
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(12, kept * size))
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": k, "score": rng.choice(["sigmoid", "softmax"]),
                "groups": groups, "kept": kept, "top2": rng.random() < 0.5, "bias": rng.random() < 0.5,
                "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5])}
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 8, 7168), "K": _log(rng, 64, 7168),
                "x": rng.choice(["bf16", "fp32"]), "y": rng.choice(["bf16", "fp32"])}
    E = _log(rng, 4, 128)
    return {"op": op, "T": _log(rng, 1, 4096), "D": 128 * _log(rng, 1, 32), "I": 128 * _log(rng, 1, 12), "E": E,
            "k": rng.randint(1, min(8, E))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _rows8(v):
    """Rows of a 32-bit tensor -> (q int8, scale fp32).  The quotient is formed in 64 bits: in 32 it falls on
    the other side of a half now and then, and a whole step of q is more than a 32-bit result allows."""
    m = v.abs().amax(dim=-1, keepdim=True)
    q = torch.where(m > 0, v.double() * 127.0 / m, 0.0)
    return torch.round(q).to(torch.int8), (m / 127.0).squeeze(-1)


def _weight(shape, g):
    """8-bit weights with a scale for each output row, from N(0, 1/fan_in)."""
    q = torch.empty(shape, dtype=torch.int8, device="cuda")
    s = torch.empty(shape[:-1], dtype=torch.float32, device="cuda")
    std = shape[-1] ** -0.5
    for i in range(shape[0]) if len(shape) == 3 else [...]:
        q[i], s[i] = _rows8(torch.randn(shape[-2:], generator=g, device="cuda") * std)
    return q, s


def _acts(T, D, g):
    """Hidden states: normal, with channels of different sizes, some of them large."""
    ch = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    return torch.randn((T, D), generator=g, device="cuda") * ch


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        st = {"logits": torch.randn((T, E), generator=g, device="cuda")}
        st["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        if op == "route_grad":
            st["dgate"] = torch.randn((T, k), generator=g, device="cuda")
            st["idx"] = _choose(_scores(st["logits"], case), st["bias"], case)
        return st
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        x = _acts(M, K, g).to(DT[case["x"]])
        q, s = _weight((N, K), g)
        wq = torch.zeros((N, (K + 127) // 128 * 128), dtype=torch.int8, device="cuda")
        wq[:, :K] = q
        return {"x": x, "wq": wq, "ws": s}
    T, D, I, E, k = (case[n] for n in ("T", "D", "I", "E", "k"))
    st = {"x": _acts(T, D, g).to(torch.bfloat16)}
    top = torch.sort(torch.randn((T, E), generator=g, device="cuda"), dim=-1, descending=True, stable=True)
    st["idx"] = top.indices[:, :k].to(torch.int32).contiguous()
    st["gate"] = torch.softmax(top.values[:, :k], dim=-1).contiguous()
    w = {}
    for n, shape in (("gate", (I, D)), ("up", (I, D)), ("down", (D, I))):
        w["q_" + n], w["s_" + n] = _weight((E,) + shape, g)
        w["qs_" + n], w["ss_" + n] = _weight(shape, g)
    st["w"] = w
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        from mixture_experts_layer_counts_amd import MoELayer, router_for, shape_for, tile_int8
        if case["op"] in ("route", "route_grad"):
            # routing from given logits does not depend on the expert widths
            st["layer"] = MoELayer(shape_for(case["T"], 128, 64, case["E"], case["k"]))
            st["router"] = router_for(score=case["score"], groups=case["groups"], kept_groups=case["kept"],
                                      group_score="top2" if case["top2"] else "max", renorm=case["renorm"],
                                      scale=case["scale"])
        elif case["op"] == "experts":
            # the routed weights are laid out once, by K planes
            for n in ("gate", "up", "down"):
                st["w"]["q_" + n] = tile_int8(st["w"]["q_" + n])
            st["layer"] = MoELayer(shape_for(case["T"], case["D"], case["I"], case["E"], case["k"],
                                             precision="int8", shared_precision="int8", weights_tiled=True))
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _scores(logits, case):
    """Scores in 64 bits: two choices next to each other differ by less than 32 bits resolve."""
    l = logits.double()
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    z = torch.exp(l - l.amax(dim=-1, keepdim=True))
    return z / z.sum(dim=-1, keepdim=True)


def _choose(s, bias, case):
    c = s if bias is None else s + bias.double()
    T, E = c.shape
    G, kept = case["groups"], case["kept"]
    if kept < G:
        gc = c.view(T, G, E // G)
        best = torch.sort(gc, dim=-1, descending=True).values
        n = 2 if case["top2"] and E // G > 1 else 1
        rank = torch.sort(best[..., :n].sum(dim=-1), dim=-1, descending=True, stable=True).indices[:, :kept]
        keep = torch.zeros((T, G), dtype=torch.bool, device=c.device)
        keep.scatter_(1, rank, True)
        c = torch.where(keep[:, :, None], gc, -math.inf).reshape(T, E)
    return torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :case["k"]].to(torch.int32)


def _gates(s, idx, case):
    w = torch.gather(s, 1, idx.long())
    if case["renorm"]:
        w = w / w.sum(dim=-1, keepdim=True)
    return w * case["scale"]


def _route(st, case):
    s = _scores(st["logits"], case)
    idx = _choose(s, st["bias"], case)
    return idx, _gates(s, idx, case).float()


def _route_grad(st, case):
    s = _scores(st["logits"], case)
    idx = st["idx"].long()
    w = torch.gather(s, 1, idx)
    dg = st["dgate"].double() * case["scale"]
    if case["renorm"]:
        W = w.sum(dim=-1, keepdim=True)
        dg = (dg - (dg * w).sum(dim=-1, keepdim=True) / W) / W
    ds = torch.zeros_like(s).scatter_(1, idx, dg)
    if case["score"] == "sigmoid":
        return (ds * s * (1.0 - s)).float()
    return (s * (ds - (ds * s).sum(dim=-1, keepdim=True))).float()


def _product(q, sx, wq, sw):
    """Integer products (exact: their sums pass 24 bits, so they are formed in 64), then the two scales."""
    return (q.double() @ wq.double().T).float() * sx[:, None] * sw[None, :]


def _linear(st, case):
    K = case["K"]
    q, sx = _rows8(st["x"].float())
    return _product(q, sx, st["wq"][:, :K], st["ws"]).to(DT[case["y"]])


def _ffn(q, sx, w, p, e=...):
    g = _product(q, sx, w["q" + p + "_gate"][e], w["s" + p + "_gate"][e])
    u = _product(q, sx, w["q" + p + "_up"][e], w["s" + p + "_up"][e])
    hq, sh = _rows8(g / (1.0 + torch.exp(-g)) * u)
    return _product(hq, sh, w["q" + p + "_down"][e], w["s" + p + "_down"][e])


def _experts(st, case):
    q, sx = _rows8(st["x"].float())
    w = st["w"]
    y = torch.zeros((case["T"], case["k"], case["D"]), dtype=torch.float32, device="cuda")
    flat = st["idx"].flatten().long()
    order = torch.sort(flat, stable=True).indices
    ends = torch.bincount(flat, minlength=case["E"]).cumsum(0).tolist()
    for e, (lo, hi) in enumerate(zip([0] + ends, ends)):
        if hi > lo:
            r = order[lo:hi]
            t = r // case["k"]
            y.view(-1, case["D"])[r] = _ffn(q[t], sx[t], w, "", e)
    out = (y * st["gate"][:, :, None]).sum(dim=1) + _ffn(q, sx, w, "s")
    return out.to(torch.bfloat16)


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"route": _route, "route_grad": _route_grad, "linear": _linear, "experts": _experts}[op](state, case)
    if op == "route":
        _, idx, gate = state["layer"].route(None, None, state["logits"], router=state["router"], bias=state["bias"])
        return idx, gate
    if op == "route_grad":
        return state["layer"].route_backward(state["logits"], state["idx"], state["dgate"], router=state["router"])
    if op == "linear":
        from mixture_experts_layer_counts_amd import linear_int8
        return linear_int8(state["x"], state["wq"], state["ws"], out_dtype=DT[case["y"]])
    layer = state["layer"]
    sched = layer.schedule(state["idx"])
    out, _ = layer.forward(state["w"], state["x"], state["x"], state["gate"], sched, out32=False)
    return out


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
    if op == "route_grad":
        T, E, k = case["T"], case["E"], case["k"]
        # softmax scores, and their gradient where it reaches every expert, need the whole row of logits
        read = k if case["score"] == "sigmoid" or case["renorm"] else E
        return {"bytes": 4 * T * read + 8 * T * k + 4 * T * E, "flops": 8 * T * read}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        ex, ey = (4 if case[n] == "fp32" else 2 for n in "xy")
        return {"bytes": ex * M * K + N * K + 4 * N + ey * M * N, "flops": 2 * M * N * K}
    T, D, I, E, k = (case[n] for n in ("T", "D", "I", "E", "k"))
    touched = E * (1.0 - (1.0 - k / E) ** T) + 1
    return {"bytes": int(touched * (3 * D * I + 4 * (2 * I + D)) + 4 * T * D + 8 * T * k),
            "flops": 6 * T * (k + 1) * D * I}


def _np_scores(l, case):
    if case["score"] == "sigmoid":
        return np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
    z = np.exp(l - l.max(axis=1, keepdims=True))
    return z / z.sum(axis=1, keepdims=True)


def _exact_route(st, case):
    s = _np_scores(st["logits"].cpu().numpy().astype(np.float64), case)
    c = s if st["bias"] is None else s + st["bias"].cpu().numpy().astype(np.float64)
    T, E = s.shape
    G = case["groups"]
    size = E // G
    if case["kept"] < G:
        part = np.sort(c.reshape(T, G, size), axis=2)
        rank = part[:, :, -1] + (part[:, :, -2] if case["top2"] and size > 1 else 0.0)
        best = np.argsort(-rank, axis=1, kind="stable")[:, :case["kept"]]
        allowed = (np.arange(E)[None, None, :] // size == best[:, :, None]).any(axis=1)
        c = np.where(allowed, c, -np.inf)
    idx = np.argsort(-c, axis=1, kind="stable")[:, :case["k"]]
    w = np.take_along_axis(s, idx, axis=1)
    gate = case["scale"] * (w / w.sum(axis=1, keepdims=True) if case["renorm"] else w)
    return idx.astype(np.int32), gate


def _exact_route_grad(st, case):
    """Through the Jacobian of the gates with respect to the logits, entry by entry."""
    s = _np_scores(st["logits"].cpu().numpy().astype(np.float64), case)
    idx = st["idx"].cpu().numpy().astype(np.int64)
    dg = st["dgate"].cpu().numpy().astype(np.float64)
    T, E = s.shape
    w = np.take_along_axis(s, idx, axis=1)
    k = idx.shape[1]
    rows = np.arange(T)
    out = np.zeros_like(s)
    if case["renorm"]:
        W = w.sum(axis=1)
        J = np.eye(k)[None] / W[:, None, None] - w[:, :, None] / (W ** 2)[:, None, None]  # dgate_i / ds_j
    else:
        J = np.broadcast_to(np.eye(k), (T, k, k))
    dw = case["scale"] * (dg[:, :, None] * J).sum(axis=1)
    for j in range(k):
        sj = w[:, j]
        if case["score"] == "sigmoid":
            out[rows, idx[:, j]] += dw[:, j] * sj * (1.0 - sj)
        else:
            row = -s * sj[:, None]
            row[rows, idx[:, j]] += sj
            out += dw[:, j:j + 1] * row
    return out


def _deq(v):
    """The values that the 8-bit form of 64-bit rows stands for."""
    m = v.abs().amax(dim=1, keepdim=True)
    q = torch.round(127.0 * v / torch.where(m > 0, m, 1.0))
    return q * (m / 127.0)


def _exact_linear(st, case):
    w = st["wq"][:, :case["K"]].double() * st["ws"].double()[:, None]
    return _deq(st["x"].double()) @ w.T


def _exact_ffn(xd, w, p, e):
    def mat(n):
        return w["q" + p + "_" + n][e].double() * w["s" + p + "_" + n][e].double()[:, None]
    g = xd @ mat("gate").T
    return _deq(g * torch.sigmoid(g) * (xd @ mat("up").T)) @ mat("down").T


def _exact_experts(st, case):
    xd = _deq(st["x"].double())
    out = _exact_ffn(xd, st["w"], "s", ...)
    idx, gate = st["idx"].long(), st["gate"].double()
    for e in torch.unique(idx).tolist():
        t, slot = torch.nonzero(idx == e, as_tuple=True)  # a token names an expert once at most
        out[t] += gate[t, slot][:, None] * _exact_ffn(xd[t], st["w"], "", e)
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    with torch.no_grad():
        return {"route": _exact_route, "route_grad": _exact_route_grad, "linear": _exact_linear,
                "experts": _exact_experts}[op](st, case)
