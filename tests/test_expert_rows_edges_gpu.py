"""The operators around a dispatch's rows in calls at the edge of what is allowed, or past it: prefixes that
descend, outputs as torch allocates them, sums over so many rows that one wait for them outlasts a short limit, and waits
that run out in the norm's gradient."""
from __future__ import annotations

import time

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


# ------------------------------------------------------------------ what allocates an output

@pytest.fixture
def deterministic():
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


def some_rows(gen, M, K, N):
    """Rows of which the first and last belong to no expert."""
    prefix = torch.tensor([2, 5, M - 3], dtype=torch.int32, device=DEV)
    return normal(gen, M, K), normal(gen, 2, N, K), prefix


def test_outputs_are_filled_as_torch_fills_them(moe, deterministic):
    """With deterministic algorithms torch.empty holds NaN: rows that a call does not write show it."""
    gen = torch.Generator(DEV).manual_seed(22)
    x, w, prefix = some_rows(gen, 40, 64, 72)
    free = [0, 1, 37, 38, 39]
    for dirty in (normal(gen, 40, 72), normal(gen, 40, 64)):   # memory that the allocator gives out again
        del dirty
    out = moe.moe_grouped_linear(x, w, prefix)
    gx = moe.moe_grouped_linear_grad_x(out.nan_to_num(), w, prefix)
    h, _ = moe.moe_swiglu(x, num_rows=torch.tensor([37], dtype=torch.int32, device=DEV))
    assert out[free].isnan().all() and out[2:37].isfinite().all()
    assert gx[free].isnan().all() and gx[2:37].isfinite().all()
    assert h[37:].isnan().all() and h[:37].isfinite().all()
    torch.utils.deterministic.fill_uninitialized_memory = False
    try:
        assert torch.equal(moe.moe_grouped_linear(x, w, prefix)[2:37], out[2:37])
    finally:
        torch.utils.deterministic.fill_uninitialized_memory = True


def test_dispatch_modes_see_outputs(moe):
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.made = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if "empty" in str(func):
                self.made.append(tuple(args[0]))
            return func(*args, **(kwargs or {}))

    gen = torch.Generator(DEV).manual_seed(23)
    x, w, prefix = some_rows(gen, 40, 64, 72)
    status, logits = moe.new_status(), torch.randn(3, 8, device=DEV, generator=gen)
    with Seen() as seen:
        moe.moe_grouped_linear(x, w, prefix, status=status)
        moe.moe_swiglu(x, status=status)
        moe.moe_add_rms_norm(x, normal(gen, 64), residual=x, status=status)
        moe.moe_topk_gate(logits, 2, status=status)
    assert [s for s in seen.made if s != (64,)] == [(40, 72), (40, 32), (40, 64), (40, 64), (3, 2), (3, 2)]


def test_outputs_in_inference_mode(moe):
    gen = torch.Generator(DEV).manual_seed(24)
    x, w, prefix = some_rows(gen, 40, 64, 72)
    with torch.inference_mode():
        assert moe.moe_grouped_linear(x, w, prefix).is_inference()
    assert not moe.moe_grouped_linear(x, w, prefix).is_inference()


def test_outputs_on_the_given_stream_with_deterministic_algorithms(moe, deterministic):
    gen = torch.Generator(DEV).manual_seed(25)
    x, w, prefix = some_rows(gen, 40, 64, 72)
    want = moe.moe_grouped_linear(x, w, prefix)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):   # the fill goes before the call on the call's stream
        got = moe.moe_grouped_linear(x, w, prefix, stream=side)
        side.synchronize()
        assert torch.equal(got[2:37], want[2:37]) and got[:2].isnan().all()


# ------------------------------------------------------------------ long reductions

@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("rows", [2 ** 25, 2 ** 25 - 4])
def test_a_long_sum_of_one_expert_is_waited_for(moe, dtype, rows):
    """2^25 rows of one expert among many take some 130 ms; a limit of 40 ms holds for each 2^22 of them. Rows of ones: sums
    up to 2^24 are whole numbers of 24 bits, beyond that they grow by 16 and at last by 16 or 12, all of them multiples of 4
    where fp32 holds multiples of 2."""
    M = 2 ** 25
    x, g = (torch.ones(M, 8, dtype=BF, device=DEV) for _ in range(2))
    prefix = torch.zeros(161, dtype=torch.int32, device=DEV)
    prefix[40:] = rows
    status = moe.new_status()
    with moe.test_wait_limits(40_000_000):
        got = moe.moe_grouped_linear_grad_w(g, x, prefix, dtype=dtype, status=status)
        torch.cuda.synchronize()
    moe.check_status(status)
    want = torch.zeros(160, 8, 8, device=DEV)
    want[39] = rows
    assert torch.equal(got, want.to(dtype))


# ------------------------------------------------------------------ waits that run out

# one group of warps to a CTA and several, one warp to a row, rows for one stage and for many rounds of the ring
@pytest.mark.parametrize("T,H", [(1, 64), (5, 16384), (1300, 16384), (1000, 14336), (3000, 7168), (9000, 1000), (40000, 256)])
@pytest.mark.parametrize("cta", [0, 3])
def test_the_norms_gradient_gives_up(moe, T, H, cta):
    """A CTA that does not fetch its first rows reports the timeout and ends, with none of its other rows on their way."""
    gen = torch.Generator(DEV).manual_seed(26)
    x, w, g, gr = normal(gen, T, H), normal(gen, H), normal(gen, T, H), normal(gen, T, H)
    status = moe.new_status()
    want = moe.moe_add_rms_norm_backward(x, w, g, grad_residual=gr, status=status)
    moe.check_status(status)
    torch.cuda.synchronize()
    with moe.test_wait_limits(20_000_000, cta):
        start = time.monotonic()
        moe.moe_add_rms_norm_backward(x, w, g, grad_residual=gr, status=status)
        torch.cuda.synchronize()
        took = time.monotonic() - start
    assert int(status.item()) == (moe.MOE_ERR_TIMEOUT if T > cta else moe.MOE_OK)
    assert took < 0.5   # a wait and one more for the rows on their way, of 20 ms each
    status.zero_()
    got = moe.moe_add_rms_norm_backward(x, w, g, grad_residual=gr, status=status)
    moe.check_status(status)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_withheld_cta_of_a_long_sum_ends_soon(moe):
    """Of the waits of a CTA that gives up, only those for a whole tile have the longer limit of many rows, 100 ms here; the
    six or seven for its copies under way have 20."""
    M = 2 ** 24
    x, g = (torch.ones(M, 256, dtype=BF, device=DEV) for _ in range(2))
    prefix = torch.full((161,), M, dtype=torch.int32, device=DEV)
    prefix[0] = 0
    status = moe.new_status()
    out = torch.empty(160, 256, 256, device=DEV)
    moe.moe_grouped_linear_grad_w(g, x, prefix, out=out, status=status)
    moe.check_status(status)
    torch.cuda.synchronize()
    with moe.test_wait_limits(20_000_000, 1):
        start = time.monotonic()
        moe.moe_grouped_linear_grad_w(g, x, prefix, out=out, status=status)
        torch.cuda.synchronize()
        took = time.monotonic() - start
    assert int(status.item()) == moe.MOE_ERR_TIMEOUT
    assert took < 0.45, took
