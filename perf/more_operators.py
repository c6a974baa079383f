"""Measured operators: a whole mixture-of-experts layer for a few tokens, and
the norms, gate, dropout and residual sum around such a layer, with their
gradient.

``run`` computes one pass of a case's operator, as elementary torch operations
or, with ``own`` set, through this framework's public calls.

Definitions:

* few: the layer from the tokens x to its output, as a step of serving runs it.
  logits l = x W_r^T; scores s = sigmoid(l), or softmax(l) over the experts;
  with groups, a group of consecutive experts ranks by the sum of its two
  largest c = s + bias (or by its largest), the best ``kept`` groups stay, and
  the k largest c among them are chosen, ties to the lower index; gates are
  ``scale`` times the chosen s, divided by their sum where ``renorm`` is set.
  out = sum_s g_s f_s(x) + f_shared(x), f(x) = W_down h,
  h = SiLU(W_gate x) * (W_up x).
  In MXFP8 the routed experts' weights, x and h are blocks of 32 values of
  E4M3 that share a power of two, X = floor(log2 max|v|) - 8; the shared expert
  stays in bf16.
* norm: z = x + scale * gate * drop(N(y) (w_post + offset)),
  h = N(z) (w_pre + offset), N(v) = v / sqrt(mean(v^2) + eps); each of the
  weights and the gate may be absent, gate [G, D] serves T / G rows each.
  drop keeps an element where its 32 random bits are at least p 2^32 and
  divides what it keeps by 1 - p.  The bits of element (t, d) are word d % 4 of
  the Philox-4x32 generator of ten rounds (Salmon et al., "Parallel random
  numbers: as easy as 1, 2, 3", 2011) at the counter (d / 4, t, offset's low
  and high word) under the key (seed's low and high word).
* norm_grad: the gradients of norm with respect to x, y, the weights and the
  gate, for given gradients of z and h, from z as the forward stored it.
"""

import math

import torch

own = False

# the sizes of one layer: hidden width, expert width, experts, experts a token
LARGE = {"D": 7168, "I": 2048, "Is": 2048, "E": 256, "k": 8}
MID = {"D": 2048, "I": 768, "Is": 768, "E": 128, "k": 8}
SIG = {"score": "sigmoid", "groups": 8, "kept": 4, "top2": True, "bias": True, "renorm": True, "scale": 2.5}
SOFT = {"score": "softmax", "groups": 1, "kept": 1, "top2": False, "bias": False, "renorm": True, "scale": 1.0}
EPS = 1e-6


def listed():
    return [
        # one token of a serving step at the middle layer: latency
        {"name": "few_t1_mid", "op": "few", "T": 1, **MID, **SOFT, "prec": "bf16", "tiled": False},
        # one token of the large layer with its grouped sigmoid router
        {"name": "few_t1", "op": "few", "T": 1, **LARGE, **SIG, "prec": "bf16", "tiled": False},
        # the same with 384 experts in MXFP8
        {"name": "few_t1_mxfp8", "op": "few", "T": 1, **{**LARGE, "E": 384}, **SOFT, "prec": "mxfp8", "tiled": True},
        # a draft of thirteen tokens through a layer of odd widths
        {"name": "few_t13", "op": "few", "T": 13, "D": 1472, "I": 320, "Is": 704, "E": 100, "k": 6, **SOFT,
         "prec": "bf16", "tiled": False},
        # a batch of eight sequences: some sixty experts
        {"name": "few_t8", "op": "few", "T": 8, **LARGE, **SIG, "prec": "bf16", "tiled": True},
        # a batch of 64 sequences: nearly every expert, several tokens each
        {"name": "few_t64_mid", "op": "few", "T": 64, **MID, **SOFT, "prec": "bf16", "tiled": True},
        {"name": "few_t64_mid_mxfp8", "op": "few", "T": 64, **MID, **SOFT, "prec": "mxfp8", "tiled": True},
        # one token between two blocks of the large model: latency
        {"name": "norm_t1", "op": "norm", "T": 1, "D": 7168, "x": "bf16", "y": "bf16", "w": "bf16", "post": True,
         "G": 0, "pre": True, "p": 0.0, "scale": 1.0, "offset": 0.0},
        # a ragged training batch with a learned gate per channel and dropout
        {"name": "norm_t4099", "op": "norm", "T": 4099, "D": 2048, "x": "bf16", "y": "bf16", "w": "bf16",
         "post": True, "G": 1, "pre": True, "p": 0.1, "scale": 0.22, "offset": 1.0},
        # a training batch or a long prompt of the large model, the stream in 32 bits
        {"name": "norm_t8192", "op": "norm", "T": 8192, "D": 7168, "x": "fp32", "y": "bf16", "w": "bf16",
         "post": True, "G": 1, "pre": True, "p": 0.0, "scale": 1.0, "offset": 0.0},
        # odd sizes, everything in 32 bits, a gate per sequence of a batch of seven
        {"name": "norm_grad_t777", "op": "norm_grad", "T": 777, "D": 1001, "x": "fp32", "y": "fp32", "w": "fp32",
         "dh": "fp32", "post": True, "G": 7, "pre": True, "p": 0.1, "scale": 0.5, "offset": 0.0},
        # the large model's training batch: dh as the layer's backward leaves it, in 32 bits
        {"name": "norm_grad_t8192", "op": "norm_grad", "T": 8192, "D": 7168, "x": "bf16", "y": "bf16", "w": "bf16",
         "dh": "fp32", "post": True, "G": 1, "pre": True, "p": 0.1, "scale": 1.0, "offset": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "norm", "norm_grad"])
    if op == "few":
        prec = rng.choice(["bf16", "bf16", "mxfp8"])
        unit = 64 if prec == "bf16" else 128
        while True:
            groups = rng.choice([1, 1, 2, 4, 8])
            E = groups * _log(rng, 2, 384 // groups)
            kept = rng.randint(max(1, groups // 2), groups)
            c = {"op": op, "T": _log(rng, 1, 64), "D": unit * _log(rng, 1, 7168 // unit),
                 "I": unit * _log(rng, 1, 2048 // unit), "Is": unit * _log(rng, 1, 4096 // unit), "E": E,
                 "k": rng.randint(1, min(12, kept * (E // groups))), "score": rng.choice(["sigmoid", "softmax"]),
                 "groups": groups, "kept": kept, "top2": rng.random() < 0.5, "bias": rng.random() < 0.5,
                 "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]), "prec": prec,
                 "tiled": rng.random() < 0.5}
            one = 3 * c["D"] * c["I"]
            # no more weights than the batch of eight at the large layer reads, and than its layer holds
            if c["T"] * c["k"] * one <= 2.8e9 and E * one <= 1.1e10:
                return c
    p = rng.choice([0.0, 0.0, 0.1, 0.25])
    T, D = _log(rng, 1, 8192), _log(rng, 32, 7168)
    G = rng.choice([0, 1, 1, max(g for g in range(1, min(T, 32) + 1) if T % g == 0)])
    c = {"op": op, "T": T, "D": D, "x": rng.choice(["bf16", "fp32"]), "y": rng.choice(["bf16", "fp32"]),
         "w": rng.choice(["bf16", "fp32"]), "post": rng.random() < 0.7, "G": G, "pre": rng.random() < 0.8, "p": p,
         "scale": rng.choice([1.0, 0.22]), "offset": rng.choice([0.0, 1.0])}
    if op == "norm_grad":
        c["dh"] = rng.choice(["bf16", "fp32"])
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _mx(v):
    """Rows of a 32-bit tensor -> (E4M3 bytes, one E8M0 byte for 32 values)."""
    b = v.unflatten(-1, (-1, 32))
    m = b.abs().amax(dim=-1, keepdim=True)
    X = torch.where(m > 0, torch.frexp(m).exponent - 9, -127).clamp(-127, 127)  # floor(log2 m) - 8
    q = torch.ldexp(b, -X).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).flatten(-2), (X + 127).to(torch.uint8).squeeze(-1)


def _mx_values(q, s):
    """What the bytes stand for, in 32 bits."""
    v = q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return torch.ldexp(v, s.int().unsqueeze(-1) - 127).flatten(-2)


def _acts(T, D, g):
    """Hidden states: normal, with channels of different sizes, some of them large."""
    ch = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    return torch.randn((T, D), generator=g, device="cuda") * ch


def _few_inputs(case, g):
    T, D, I, Is, E = (case[n] for n in ("T", "D", "I", "Is", "E"))
    st = {"x": (_acts(T, D, g) * 0.88).to(torch.bfloat16)}
    st["w_router"] = (torch.randn((E, D), generator=g, device="cuda") * D ** -0.5).to(torch.bfloat16)
    st["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
    w = {}
    for n, N, K in (("gate", I, D), ("up", I, D), ("down", D, I)):
        if case["prec"] == "bf16":
            w["w_" + n] = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
        else:
            w["q_" + n] = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
            w["s_" + n] = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
        for e in range(E):
            m = torch.randn((N, K), generator=g, device="cuda") * K ** -0.5
            if case["prec"] == "bf16":
                w["w_" + n][e] = m
            else:
                w["q_" + n][e], w["s_" + n][e] = _mx(m)
    for n, N, K in (("gate", Is, D), ("up", Is, D), ("down", D, Is)):
        w["ws_" + n] = (torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    st["w"] = w
    return st


def _norm_inputs(case, g):
    T, D, G = case["T"], case["D"], case["G"]
    st = {"x": _acts(T, D, g).to(DT[case["x"]]), "y": _acts(T, D, g).to(DT[case["y"]])}

    def near_one(*shape):
        return (1.0 - case["offset"] + 0.2 * torch.randn(shape, generator=g, device="cuda")).to(DT[case["w"]])
    st["post"] = near_one(D) if case["post"] else None
    st["pre"] = near_one(D) if case["pre"] else None
    st["gate"] = torch.randn((G, D), generator=g, device="cuda").to(DT[case["w"]]) if G else None
    st["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda") if case["p"] else None
    if case["op"] == "norm_grad":  # x's place is z's: the stream as the forward stored it
        st["dz"] = torch.randn((T, D), generator=g, device="cuda").to(DT[case["x"]])
        st["dh"] = torch.randn((T, D), generator=g, device="cuda").to(DT[case["dh"]]) if case["pre"] else None
    return st


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _few_inputs(case, g) if case["op"] == "few" else _norm_inputs(case, g)


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own and case["op"] == "few":
        from mixture_experts_layer_counts_amd import (MoELayer, pack_mxfp8_scales, router_for, shape_for, tile_bf16,
                                                      tile_mxfp8)
        w = st["w"]
        for n in ("gate", "up", "down"):  # the weights are laid out once
            if case["prec"] == "mxfp8":
                w["s_" + n] = pack_mxfp8_scales(w["s_" + n])
                w["q_" + n] = tile_mxfp8(w["q_" + n]) if case["tiled"] else w["q_" + n]
            elif case["tiled"]:
                w["w_" + n] = tile_bf16(w["w_" + n])
        st["layer"] = MoELayer(shape_for(case["T"], case["D"], case["I"], case["E"], case["k"], I_shared=case["Is"],
                                         precision=case["prec"], weights_tiled=case["tiled"]))
        st["router"] = router_for(score=case["score"], groups=case["groups"], kept_groups=case["kept"],
                                  group_score="top2" if case["top2"] else "max", renorm=case["renorm"],
                                  scale=case["scale"])
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _scores(l, case):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    z = torch.exp(l - l.amax(dim=-1, keepdim=True))
    return z / z.sum(dim=-1, keepdim=True)


def _route(x, w_router, bias, case):
    """Scores in 64 bits: two choices next to each other differ by less than 32 bits resolve."""
    l = x.double() @ w_router.double().T
    s = _scores(l, case)
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
    idx = torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :case["k"]]
    w = torch.gather(s, 1, idx)
    if case["renorm"]:
        w = w / w.sum(dim=-1, keepdim=True)
    return l.float(), idx.to(torch.int32), (w * case["scale"]).float()


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _few(st, case):
    x, w = st["x"], st["w"]
    logits, idx, gate = _route(x, st["w_router"], st["bias"], case)
    e = idx.flatten().long()
    rows = x.float().repeat_interleave(case["k"], dim=0).unsqueeze(-1)  # [T k, D, 1]
    if case["prec"] == "bf16":
        def product(n, v):
            return w["w_" + n][e].float() @ v
    else:
        def product(n, v):
            return _mx_values(w["q_" + n][e], w["s_" + n][e]) @ _mx_values(*_mx(v.squeeze(-1))).unsqueeze(-1)
    h = _silu(product("gate", rows)) * product("up", rows)
    y = product("down", h).view(case["T"], case["k"], case["D"])
    x32 = x.float()
    hs = _silu(x32 @ w["ws_gate"].float().T) * (x32 @ w["ws_up"].float().T)
    out = (y * gate[:, :, None]).sum(dim=1) + hs @ w["ws_down"].float().T
    return logits, idx, gate, out.to(torch.bfloat16)


M32 = 0xFFFFFFFF


def _philox_round(c, k):
    a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64-bit products, wrapped: their words are right
    return ((b >> 32) & M32) ^ c[1] ^ k[0], b & M32, ((a >> 32) & M32) ^ c[3] ^ k[1], a & M32


def _kept(T, D, p, rng):
    """The elements that dropout keeps."""
    quads = (D + 3) // 4
    seed, offset = rng[0], rng[1]
    c = (torch.arange(quads, device="cuda").expand(T, quads), torch.arange(T, device="cuda")[:, None],
         offset & M32, (offset >> 32) & M32)
    k = (seed & M32, (seed >> 32) & M32)
    for r in range(10):
        c = _philox_round(c, ((k[0] + r * 0x9E3779B9) & M32, (k[1] + r * 0xBB67AE85) & M32))
    bits = torch.stack(torch.broadcast_tensors(*c), dim=-1).reshape(T, 4 * quads)[:, :D]
    return bits >= round(p * 2 ** 32)


def _rows(gate, T):
    return gate.float().repeat_interleave(T // gate.shape[0], dim=0)


def _factor(st, case):
    """What N(y) (w_post + offset) is multiplied by."""
    T, D = case["T"], case["D"]
    f = case["scale"]
    if case["p"]:
        f = _kept(T, D, case["p"], st["rng"]).float() * (f / (1.0 - case["p"]))
    return f


def _norm(st, case):
    z, y = st["x"].float(), st["y"].float()
    if st["post"] is not None:
        y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS) * (st["post"].float() + case["offset"])
    if st["gate"] is not None:
        y = y * _rows(st["gate"], case["T"])
    z = z + y * _factor(st, case)
    out = [z.to(DT[case["x"]])]
    if st["pre"] is not None:
        h = z * torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + EPS) * (st["pre"].float() + case["offset"])
        out.append(h.to(torch.bfloat16))
    return out


def _norm_grad(st, case):
    T, D = case["T"], case["D"]
    z, y, dz = st["x"].float(), st["y"].float(), st["dz"].float()
    out = {}
    if st["pre"] is not None:
        r = torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + EPS)
        dh = st["dh"].float()
        out["dpre"] = (dh * z * r).sum(dim=0)
        v = dh * (st["pre"].float() + case["offset"])
        dz = dz + r * (v - z * r * ((v * z).mean(dim=-1, keepdim=True) * r))
    out["dx"] = dz.to(DT[case["x"]])
    dn = dz * _factor(st, case)
    r, n = 1.0, y
    if st["post"] is not None:
        r = torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS)
        n = y * r * (st["post"].float() + case["offset"])
    if st["gate"] is not None:
        G = case["G"]
        out["dgate"] = (dn * n).view(G, T // G, D).sum(dim=1)
        dn = dn * _rows(st["gate"], T)
    if st["post"] is not None:
        out["dpost"] = (dn * y * r).sum(dim=0)
        v = dn * (st["post"].float() + case["offset"])
        dn = r * (v - y * r * ((v * y).mean(dim=-1, keepdim=True) * r))
    out["dy"] = dn.to(DT[case["y"]])
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"few": _few, "norm": _norm, "norm_grad": _norm_grad}[op](state, case)
    if op == "few":
        r = state["layer"].few(state["x"], state["w_router"], state["w"], router=state["router"],
                               bias=state["bias"], out32=False)
        return r["logits"], r["idx"], r["gate"], r["out"]
    from mixture_experts_layer_counts_amd import block_norm, block_norm_backward
    opts = {"post_weight": state["post"], "gate": state["gate"], "pre_weight": state["pre"], "scale": case["scale"],
            "weight_offset": case["offset"], "eps": EPS, "dropout": case["p"], "rng": state["rng"]}
    if op == "norm":
        z, h = block_norm(state["x"], state["y"], **opts)
        return [z] if h is None else [z, h]
    g = block_norm_backward(state["x"], state["y"], state["dz"], state["dh"], **opts)
    names = {"dpre": "dpre_weight", "dx": "dx", "dgate": "dgate", "dpost": "dpost_weight", "dy": "dy"}
    return {n: g[m] for n, m in names.items() if g[m] is not None}


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------
def work(case):
    T, D = case["T"], case["D"]
    if case["op"] == "few":
        I, Is, E, k = (case[n] for n in ("I", "Is", "E", "k"))
        touched = E * (1.0 - (1.0 - k / E) ** T)
        weight = 2.0 if case["prec"] == "bf16" else 1.0 + 1.0 / 32
        return {"bytes": int(touched * 3 * D * I * weight + 6 * D * Is + 2 * E * D + 4 * T * D + 4 * T * E + 8 * T * k),
                "flops": 6 * T * D * (k * I + Is) + 2 * T * D * E}
    b = {n: 4 if case.get(n) == "fp32" else 2 for n in ("x", "y", "w", "dh")}
    params = b["w"] * D * (case["post"] + case["pre"] + case["G"])
    if case["op"] == "norm":
        return {"bytes": T * D * (2 * b["x"] + b["y"] + 2 * case["pre"]) + params, "flops": 12 * T * D}
    grads = 4 * D * (case["post"] + case["pre"] + case["G"])
    reads = b["x"] * (1 + case["pre"]) + b["dh"] * case["pre"]  # dz, and z and dh where h is formed
    y_read = b["y"] if case["post"] or case["G"] else 0
    return {"bytes": T * D * (reads + y_read + b["x"] + b["y"]) + params + grads, "flops": 25 * T * D}


def _exact_mx(v):
    """The values that blocks of 32 of a 64-bit tensor are stored as."""
    b = v.unflatten(-1, (-1, 32))
    m = b.abs().amax(dim=-1, keepdim=True)
    X = torch.where(m > 0, torch.floor(torch.log2(torch.where(m > 0, m, 1.0))) - 8, -127.0)
    X = torch.where(torch.exp2(X + 8) > m, X - 1, torch.where(torch.exp2(X + 9) <= m, X + 1, X)).clamp(-127, 127)
    u = (b / torch.exp2(X)).clamp(-448, 448)
    _, e = torch.frexp(u)
    step = torch.exp2((e - 4).clamp(min=-9).double())  # three bits behind the leading one; 2^-9 among the smallest
    return (torch.round(u / step) * step * torch.exp2(X)).flatten(-2)


def _exact_weights(w, n, e, prec):
    if prec == "bf16":
        return w["w_" + n][e].double()
    v = w["q_" + n][e].view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
    return (v * torch.exp2(w["s_" + n][e].double() - 127).unsqueeze(-1)).flatten(-2)


def _exact_few(st, case):
    x, w, k = st["x"].double(), st["w"], case["k"]
    l = (x.cpu() @ st["w_router"].double().cpu().T)
    if case["score"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.softmax(l, dim=-1)
    c = s.clone() if st["bias"] is None else s + st["bias"].double().cpu()
    T, E = c.shape
    size = E // case["groups"]
    idx = torch.zeros((T, k), dtype=torch.int32)
    for t in range(T):
        row = c[t].tolist()
        ranks = []
        for g in range(case["groups"]):
            part = sorted(row[g * size:(g + 1) * size], reverse=True)
            ranks.append((-sum(part[:2 if case["top2"] else 1]), g))
        stay = {g for _, g in sorted(ranks)[:case["kept"]]}
        best = sorted((-v, e) for e, v in enumerate(row) if e // size in stay)[:k]
        idx[t] = torch.tensor([e for _, e in best])
    chosen = torch.gather(s, 1, idx.long())
    gate = case["scale"] * (chosen / chosen.sum(dim=1, keepdim=True) if case["renorm"] else chosen)
    quant = _exact_mx if case["prec"] == "mxfp8" else (lambda v: v)

    def ffn(v, mat, q):
        a, u = q(v) @ mat("gate").T, q(v) @ mat("up").T
        return q(a * torch.sigmoid(a) * u) @ mat("down").T
    out = ffn(x, lambda n: w["ws_" + n].double(), lambda v: v)
    where, amount = idx.to(x.device), gate.to(x.device)
    for e in torch.unique(idx).tolist():
        t, slot = torch.nonzero(where == e, as_tuple=True)  # a token names an expert once at most
        out[t] += amount[t, slot][:, None] * ffn(x[t], lambda n: _exact_weights(w, n, e, case["prec"]), quant)
    return l, idx, gate, out


def _exact_bits(T, D, rng):
    """Philox in Python's integers for the rows' counters, word by word, on 64-bit arrays of 16-bit limbs."""
    seed, offset = (int(v) for v in rng.tolist())
    quads = (D + 3) // 4

    def mul(a, m):  # the high and low words of a 32 x 32 bit product, from 16-bit halves
        al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
        mid = ah * ml + ((al * ml) >> 16)
        mid2 = al * mh + (mid & 0xFFFF)
        return ah * mh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((al * ml) & 0xFFFF)
    dev = rng.device
    x0 = torch.arange(quads, device=dev).repeat(T, 1)
    x1 = torch.arange(T, device=dev).unsqueeze(1).repeat(1, quads)
    x2 = torch.full_like(x0, offset % 2 ** 32)
    x3 = torch.full_like(x0, offset // 2 ** 32)
    k0, k1 = seed % 2 ** 32, seed // 2 ** 32
    for _ in range(10):
        h0, l0 = mul(x0, 0xD2511F53)
        h1, l1 = mul(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    out = torch.empty((T, 4 * quads), dtype=torch.int64, device=dev)
    for i, v in enumerate((x0, x1, x2, x3)):
        out[:, i::4] = v
    return out[:, :D]


def _exact_norm(st, case):
    """The forward in 64 bits; its gradients by torch's differentiation of it."""
    T, D = case["T"], case["D"]
    grad = case["op"] == "norm_grad"
    leaves = {n: st[n].double().requires_grad_(grad) for n in ("x", "y", "post", "pre", "gate") if st[n] is not None}
    n = leaves["y"]
    if "post" in leaves:
        n = n / torch.sqrt(n.square().sum(dim=1, keepdim=True) / D + EPS) * (leaves["post"] + case["offset"])
    if "gate" in leaves:
        n = (n.view(case["G"], T // case["G"], D) * leaves["gate"][:, None, :]).view(T, D)
    n = n * case["scale"]
    if case["p"]:
        n = torch.where(_exact_bits(T, D, st["rng"]) < int(case["p"] * 2.0 ** 32 + 0.5), 0.0, n / (1.0 - case["p"]))
    # for the gradient x holds z itself: the sum is formed so that its value is z and its slopes are the sum's
    z = leaves["x"] + (n - n.detach() if grad else n)
    h = None
    if "pre" in leaves:
        h = z / torch.sqrt(z.square().sum(dim=1, keepdim=True) / D + EPS) * (leaves["pre"] + case["offset"])
    if not grad:
        return [z] if h is None else [z, h]
    total = (z * st["dz"].double()).sum()
    if h is not None:
        total = total + (h * st["dh"].double()).sum()
    total.backward()
    names = {"dpre": "pre", "dx": "x", "dgate": "gate", "dpost": "post", "dy": "y"}
    return {a: leaves[b].grad for a, b in names.items() if b in leaves}


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "few":
        with torch.no_grad():
            return _exact_few(st, case)
    return _exact_norm(st, case)
