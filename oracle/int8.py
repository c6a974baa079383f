"""8-bit integer rows and the experts computed from them, in fp64 (numpy).

    m = max |v| of a row,  q = round(127 v / m) (ties to even),  scale = m / 127
    f(x) = W_down q(h),  h = SiLU(W_gate q(x)) * (W_up q(x))

A row of zeros has q = 0 and scale 0.
"""

from __future__ import annotations

from typing import Dict, Tuple

import numpy as np


def quantize(v: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(q int64, scale fp64) of the rows of v."""
    v = np.asarray(v, dtype=np.float64)
    m = np.abs(v).max(axis=-1, keepdims=True)
    # 127 v and m come from values of at most 24 bits: the quotient of two
    # such numbers is exact where it is a half
    q = np.rint(127.0 * v / np.where(m > 0, m, 1.0)).astype(np.int64)
    return q, m[..., 0] / 127.0


def product(q: np.ndarray, s: np.ndarray, wq: np.ndarray, ws: np.ndarray) -> np.ndarray:
    # integers below 2^53: exact in fp64
    return (q.astype(np.float64) @ wq.astype(np.float64).T) * s[:, None] * np.asarray(ws, dtype=np.float64)[None, :]


def ffn(x: np.ndarray, w: Dict[str, np.ndarray], prefix: str, e=None) -> Tuple[np.ndarray, np.ndarray]:
    """(f(x), m of each row of h) for rows x; weights "q{prefix}_gate" and so
    on with scales "s{prefix}_gate", of expert e when they are stacked."""
    def mat(n):
        q, s = w[f"q{prefix}_{n}"], w[f"s{prefix}_{n}"]
        return (q, s) if e is None else (q[e], s[e])
    q, s = quantize(x)
    g = product(q, s, *mat("gate"))
    h = g / (1.0 + np.exp(-g)) * product(q, s, *mat("up"))
    hq, hs = quantize(h)
    return product(hq, hs, *mat("down")), hs * 127.0
