"""moe_block_norm and its gradient where test_gpu_norm.py does not go, under its bounds: many gate rows within a run of
rows whose last chunk overlaps, and dropped values in a row that is normalised.

The bounds, counted from the kernels (u = 2^-24): a row's sums are chains of 8 or 17 additions in a thread (one or two
chunks), 6 steps over a wave and up to 16 waves one after the other, 39 u at most of the sum of absolute values and
half of it behind the root; with some twenty operations around them below 64 u. Column sums are chains over a run's
rows (a run of several groups adds their sums up, with no more additions than rows), then over a sixteenth of the
runs, then over 16: with 4096 * 64 / lanes runs at most (4096 where a wave has a row, D up to 512; 256 above 4096
columns) and two rows a run at least, T rows take ceil(T / runs) + ceil(runs / 16) + 15 additions. That comes closest
to T / 64 + 160 with 273 against 287 at T = 8161 and D up to 512 (142 against 222 at T = 4000, 281 against 785 at
40000).
"""

import pytest
import torch

from mixture_experts_layer_counts_amd import block_norm, block_norm_backward
from tests._gpu import need_gpu, say
from tests.test_gpu_norm import BF, F32, Case, check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,G,wt", [(9000, 41, 9000, F32), (16390, 23, 8195, BF), (9001, 519, 9001, BF)])
def test_many_gate_rows_a_run(T, D, G, wt):
    """A run's part of dw_post is added up group by group, by single values in the chunk that overlaps."""
    dev = need_gpu()
    say("norm, gate rows a run", T, D, G)
    c = Case(dev, T, D, F32, BF, wt, BF, True, G, True, 0.0, seed=T)
    check_forward(c)
    check_backward(c)


def test_dropped_values_without_and_with_a_norm():
    """What dropout drops adds nothing to the sum; but a row that is normalised first takes every value of it into its
    statistics, dropped or not: an infinity there leaves the row's z at x, a NaN makes its kept values NaN, and the
    row's dy is not finite.  No other row, and no dx, changes by a bit."""
    dev = need_gpu()
    inf, nan = float("inf"), float("nan")
    for post in (False, True):
        c = Case(dev, 12, 104, BF, BF, BF, BF, post, 3, True, 0.5, seed=4)
        z0, h0 = block_norm(c.x, c.y, **c.kw)
        g0 = block_norm_backward(z0, c.y, c.dz, c.dh, **c.kw)
        y = c.y.clone()
        for t, v in ((2, inf), (7, nan)):
            d = int((~c.keep[t]).nonzero()[5])
            y[t, d] = v
        z, h = block_norm(c.x, y, **c.kw)
        g = block_norm_backward(z0, y, c.dz, c.dh, **c.kw)
        rest = [t for t in range(12) if t not in (2, 7)]
        for a, b in ((z, z0), (h, h0), (g["dx"], g0["dx"]), (g["dy"], g0["dy"])):
            assert torch.equal(a[rest], b[rest])
        assert torch.equal(g["dx"], g0["dx"]) and torch.equal(g["dpre_weight"], g0["dpre_weight"])
        if not post:
            assert torch.equal(z, z0) and torch.equal(h, h0)
            assert all(torch.equal(g[n], g0[n]) for n in ("dy", "dgate"))
            continue
        assert torch.equal(z[2], c.x[2])
        keep = c.keep[7]
        assert torch.equal(z[7][~keep], c.x[7][~keep]) and bool(torch.isnan(z[7][keep]).all())
        assert not torch.isfinite(g["dy"][[2, 7]]).any()
        # gate rows 0 (tokens 0 .. 3) and 1 (4 .. 7) have such a row, row 2 has none
        assert torch.equal(g["dgate"][2], g0["dgate"][2])
