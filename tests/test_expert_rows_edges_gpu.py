"""The operators around a dispatch's rows in calls at the edge of what is allowed, or past it: prefixes that descend."""
from __future__ import annotations

import pytest
import torch

from test_grouped_gpu import BF, DEV, close, codes, normal, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


# ------------------------------------------------------------------ prefixes that are wrong

def claims(prefix, M):
    """Rows of each expert, as the header has it: inside [0, M], and from the end of the earlier experts' rows on."""
    end, rows = 0, []
    for p0, p1 in zip(prefix, prefix[1:]):
        lo = max(min(max(p0, 0), M), end)
        hi = min(max(p1, lo), M)
        rows.append(slice(lo, hi))
        end = hi if hi > lo else end
    return rows


# M, K, N, prefix. The first ones make more tiles than disjoint rows can (a cluster that shares a tile takes no other).
WRONG = {
    "claimed eight times": (2048, 7168, 128, [0, 1024] * 8 + [2048]),
    "claimed three times": (1024, 7168, 128, [0, 512] * 3 + [1024]),
    "pairs": (1500, 264, 4104, [0, 700, 100, 900, 850, 1500]),
    "one expert back": (300, 7168, 512, [0, 300, 0]),
    "behind the rows": (200, 512, 264, [0, 40, 500, 700]),
    "before them": (200, 512, 264, [-50, 40, -1, 160, 200]),
    "an empty one first": (600, 7168, 264, [400, 500, 100, 600]),
    "from chunk to chunk": (900, 1024, 136, [0] + [500] * 30 + [0, 400] + [30] * 40 + [900, 10, 20]),
    "none, then back": (700, 256, 136, [400] * 40 + [100, 600, 20, 700]),
    "far numbers": (100, 256, 136, [0, 2 ** 31 - 1, -2 ** 31, 50, 100]),
}


@pytest.mark.parametrize("name", WRONG)
def test_rows_of_a_descending_prefix(moe, name):
    """The call is reported, and its outputs are what the header says all the same."""
    M, K, N, p = WRONG[name]
    E = len(p) - 1
    gen = torch.Generator(DEV).manual_seed(21)
    prefix = torch.tensor(p, dtype=torch.int64).to(torch.int32).to(DEV)
    x, g, w = normal(gen, M, K), normal(gen, M, N), normal(gen, E, N, K, std=K ** -0.5)
    (x8, xs), (w8, ws) = (codes(gen, M, K), codes(gen, E, N, K)) if K % 128 == 0 else ((None,) * 2,) * 2
    out, gx, out8 = (torch.full((M, c), 7.0, dtype=BF, device=DEV) for c in (N, K, N))

    def reported(call):
        status = moe.new_status()
        got = call(status)
        assert int(status.item()) == moe.MOE_ERR_BAD_PREFIX
        return got

    reported(lambda s: moe.moe_grouped_linear(x, w, prefix, out=out, status=s))
    reported(lambda s: moe.moe_grouped_linear_grad_x(g, w, prefix, out=gx, status=s))
    if x8 is not None:
        reported(lambda s: moe.moe_grouped_linear(x8, w8, prefix, x_scales=xs, w_scales=ws, out=out8, status=s))
    gw = reported(lambda s: moe.moe_grouped_linear_grad_w(g, x, prefix, status=s))
    free = torch.ones(M, dtype=torch.bool)
    for e, r in enumerate(claims(p, M)):
        free[r] = False
        if r.start < r.stop:
            xe, ge, we = x[r].double(), g[r].double(), w[e].double()
            close(out[r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)
            close(gx[r], ge @ we, ge.abs() @ we.abs(), N, 2.0 ** -8)
            if x8 is not None:
                xe, we = values(x8[r], xs[r]), values(w8[e], ws[e])
                close(out8[r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)
        # a weight's gradient takes all rows that its expert claims
        lo = min(max(p[e], 0), M)
        r = slice(lo, min(max(p[e + 1], lo), M))
        xe, ge = x[r].double(), g[r].double()
        close(gw[e], ge.T @ xe, ge.abs().T @ xe.abs(), max(1, r.stop - r.start), 2.0 ** -24)
    for t in (out, gx) + ((out8,) if x8 is not None else ()):
        assert (t[free.to(DEV)] == 7).all()
