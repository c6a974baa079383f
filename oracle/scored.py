"""Routing from scores, and its gradient, in fp64 (numpy).

    s_e = 1 / (1 + exp(-l_e)),  or the softmax of the logits over all experts
    c_e = s_e + b_e
    groups rank by their largest c, or the sum of their two largest; of the
    kept ones' experts the k largest c are chosen, ties to the lower id
    g_s = scale s_s / sum s   (renormalised), or scale s_s

The bias only chooses.  A logit of -inf scores 0; a renormalised gate is 0
where every chosen logit is -inf.
"""

from __future__ import annotations

from typing import Optional

import numpy as np


def scores(logits: np.ndarray, kind: str) -> np.ndarray:
    l = np.asarray(logits, dtype=np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    m = l.max(axis=1, keepdims=True)
    z = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    total = z.sum(axis=1, keepdims=True)
    return np.divide(z, total, out=np.zeros_like(z), where=total > 0)


def choose(s: np.ndarray, bias: Optional[np.ndarray], k: int, groups: int = 1, kept: int = 1,
           group_score: str = "top2") -> np.ndarray:
    """idx [T, k] int32."""
    T, E = s.shape
    size = E // groups
    c = s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
    idx = np.zeros((T, k), dtype=np.int32)
    for t in range(T):
        allowed = range(E)
        if kept < groups:
            def rank(g):
                top = sorted(c[t, g * size:(g + 1) * size], reverse=True)
                return sum(top[:2]) if group_score == "top2" else top[0]
            best = sorted(range(groups), key=lambda g: (-rank(g), g))[:kept]
            allowed = [e for g in best for e in range(g * size, (g + 1) * size)]
        idx[t] = sorted(allowed, key=lambda e: (-c[t, e], e))[:k]
    return idx


def gates(s: np.ndarray, idx: np.ndarray, renorm: bool, scale: float) -> np.ndarray:
    w = np.take_along_axis(s, idx.astype(np.int64), axis=1)
    if renorm:
        W = w.sum(axis=1, keepdims=True)
        w = np.divide(w, W, out=np.zeros_like(w), where=W > 0)
    return scale * w


def ratios(logits: np.ndarray, idx: np.ndarray, kind: str) -> np.ndarray:
    """s_s / sum s over the chosen, from the scores' logarithms: also where the
    scores themselves are below the range of fp64."""
    l = np.take_along_axis(np.asarray(logits, dtype=np.float64), idx.astype(np.int64), axis=1)
    if kind == "sigmoid":
        l = -np.logaddexp(0.0, -l)
    m = l.max(axis=1, keepdims=True)
    z = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    W = z.sum(axis=1, keepdims=True)
    return np.divide(z, W, out=np.zeros_like(z), where=W > 0)


def backward(logits: np.ndarray, idx: np.ndarray, dgate: np.ndarray, kind: str, renorm: bool,
             scale: float) -> np.ndarray:
    """dlogits [T, E] of sum(gates * dgate), the choice held fixed."""
    logits = np.asarray(logits, dtype=np.float64)
    s = scores(logits, kind)
    idx = idx.astype(np.int64)
    dw = scale * np.asarray(dgate, dtype=np.float64)
    ds = np.zeros_like(s)
    if renorm:
        p = ratios(logits, idx, kind)
        np.put_along_axis(ds, idx, p * (dw - (dw * p).sum(axis=1, keepdims=True)), axis=1)
        return ds * scores(-logits, kind) if kind == "sigmoid" else ds
    np.put_along_axis(ds, idx, dw, axis=1)
    if kind == "sigmoid":
        return ds * s * scores(-logits, kind)  # 1 - s without its cancellation
    return s * (ds - (ds * s).sum(axis=1, keepdims=True))
