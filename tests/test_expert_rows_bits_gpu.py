"""The bits that the grouped products' sums hold, and the calls that write over their inputs.

Whole numbers whose sums stay below 2^24 are exact in fp32 in whatever order they are added, and need all of its 24 bits: a
result that kept fewer on the way would differ. Results in bf16 are then the exact sum rounded once."""
from __future__ import annotations

import pytest
import torch

from test_grouped_gpu import BF, DEV, normal, prefix_of
from test_grouped_ways_gpu import WAYS, WEIGHTS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


def numbers(gen, most, *shape):
    """Whole numbers from 1 to `most` (at most 256, which bf16 holds)."""
    return torch.randint(1, most + 1, shape, device=DEV, generator=gen).to(BF)


def largest(terms):
    """The largest whole number of which `terms` squares stay below 2^24."""
    return min(256, int(((2 ** 24 - 1) / terms) ** 0.5))


def rounded(sums):
    assert sums.max() < 2 ** 24
    return sums.float().to(BF)


@pytest.mark.parametrize("name", WAYS)
def test_sums_of_products_are_exact(moe, name):
    counts, K, N = WAYS[name]
    gen = torch.Generator(DEV).manual_seed(31)
    p = prefix_of(counts)
    M, E, status = p[-1], len(counts), moe.new_status()
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, w, g = numbers(gen, largest(K), M, K), numbers(gen, largest(max(K, N)), E, N, K), numbers(gen, largest(N), M, N)
    out = moe.moe_grouped_linear(x, w, prefix, status=status)
    gx = moe.moe_grouped_linear_grad_x(g, w, prefix, status=status)
    moe.check_status(status)
    for e in range(E):
        r = slice(p[e], p[e + 1])
        if counts[e]:
            assert torch.equal(out[r], rounded(x[r].double() @ w[e].double().T))
            assert torch.equal(gx[r], rounded(g[r].double() @ w[e].double()))


@pytest.mark.parametrize("name", WAYS)
def test_sums_of_e4m3_products_are_exact(moe, name):
    """Scales of 1/2, 1 and 2 on each side: multiples of 1/4, below 2^22."""
    counts, K, N = WAYS[name]
    K = -(-K // 128) * 128
    gen = torch.Generator(DEV).manual_seed(32)
    p = prefix_of(counts)
    M, E, most, status = p[-1], len(counts), min(16, largest(16 * K)), moe.new_status()   # E4M3 holds 1 to 16
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)

    def made(*shape):
        v = numbers(gen, most, *shape)
        s = 2.0 ** torch.randint(-1, 2, (*shape[:-1], K // 128), device=DEV, generator=gen).float()
        return v.float().to(torch.float8_e4m3fn).view(torch.uint8), s, v.double() * s.double().repeat_interleave(128, -1)

    (x, xs, x64), (w, ws, w64) = made(M, K), made(E, N, K)
    out = moe.moe_grouped_linear(x, w, prefix, x_scales=xs, w_scales=ws, status=status)
    moe.check_status(status)
    for e in range(E):
        r = slice(p[e], p[e + 1])
        if counts[e]:
            assert torch.equal(out[r], rounded(x64[r] @ w64[e].T))


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("name", WEIGHTS)
def test_sums_of_rows_are_exact(moe, name, dtype):
    """Written, and added in fp32 to whole numbers. (What bf16 holds before would take the sum past 24 bits' rounding.)"""
    counts, K, N = WEIGHTS[name]
    gen = torch.Generator(DEV).manual_seed(33)
    p = prefix_of(counts, 3)
    M, E, most, status = p[-1] + 5, len(counts), largest(max(counts) + 1), moe.new_status()
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, g = numbers(gen, most, M, K), numbers(gen, most, M, N)
    start = torch.randint(0, most * most + 1, (E, N, K), device=DEV, generator=gen).float()
    out = moe.moe_grouped_linear_grad_w(g, x, prefix, dtype=dtype, status=status)
    added = moe.moe_grouped_linear_grad_w(g, x, prefix, out=start.clone(), accumulate=True, status=status)
    moe.check_status(status)
    for e in range(E):
        want = g[p[e]: p[e + 1]].double().T @ x[p[e]: p[e + 1]].double()
        assert want.max() + start.max() < 2 ** 24
        assert torch.equal(out[e], want.float().to(dtype))
        assert torch.equal(added[e].double(), want + start[e].double())


# ------------------------------------------------------------------ in place

# one pass over a row's channels and several; several rows to a CTA and one; rows for many turns of the grid
@pytest.mark.parametrize("M,I", [(1, 8), (9000, 264), (3000, 1416), (1500, 12296)])
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu_backward_over_its_input(moe, M, I, weighted):
    gen = torch.Generator(DEV).manual_seed(34)
    gu, g = normal(gen, M, 2 * I), normal(gen, M, I)
    w = torch.rand(M, device=DEV, generator=gen) if weighted else None
    want, want_w = moe.moe_swiglu_backward(gu, g, row_weights=w)
    got, got_w = moe.moe_swiglu_backward(gu, g, row_weights=w, out=gu)
    assert got.data_ptr() == gu.data_ptr() and torch.equal(got, want)
    assert want_w is None or torch.equal(got_w, want_w)


SIZES = [(1, 8), (40000, 256), (9000, 1000), (4000, 7168), (2000, 14336), (2000, 16384)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("over", ["h", "grad", "grad_residual"])
def test_norm_backward_over_an_input(moe, T, H, over):
    """Rows are fetched ahead, many more of them than a CTA's ring holds."""
    gen = torch.Generator(DEV).manual_seed(35)
    t = dict(h=normal(gen, T, H), grad=normal(gen, T, H), grad_residual=normal(gen, T, H))
    w = normal(gen, H)
    want = moe.moe_add_rms_norm_backward(t["h"], w, t["grad"], grad_residual=t["grad_residual"])
    got = moe.moe_add_rms_norm_backward(t["h"], w, t["grad"], grad_residual=t["grad_residual"], out=t[over])
    assert got[0].data_ptr() == t[over].data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("over", ["x", "residual"])
def test_norm_over_an_input(moe, T, H, over):
    gen = torch.Generator(DEV).manual_seed(36)
    t = dict(x=normal(gen, T, H), residual=normal(gen, T, H))
    w, codes = normal(gen, H), H % 128 == 0
    want = moe.moe_add_rms_norm(t["x"], w, residual=t["residual"], quantize_fp8=codes)
    got = moe.moe_add_rms_norm(t["x"], w, residual=t["residual"], quantize_fp8=codes, residual_out=t[over])
    assert got.residual.data_ptr() == t[over].data_ptr()
    for a, b in ((got.out, want.out), (got.residual, want.residual), (got.codes, want.codes), (got.scales, want.scales)):
        assert (a is None and b is None) or torch.equal(a, b)
