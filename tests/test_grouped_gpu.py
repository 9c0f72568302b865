"""moe_grouped_linear and its gradients against their formulas in 64 bits.

Tolerances. Products of two bf16 (or two E4M3 codes) are exact in fp32. A sum of K of them is rounded, or cut, once for
each instruction of 16 (32) products and at most once for each product while these are aligned: at most K/16 + 16 errors
of 2^-23 of the sum of magnitudes S so far. A result in bf16 adds half a step, 2^-8 of it, one in fp32 2^-24. With E4M3
each block of 128 is then multiplied by its scales and added: K/128 more steps with three roundings of 2^-24 each, fewer
than those already counted."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


# rows of each expert: none, one, around a tensor-core step, around tiles of 32 to 256, several tiles
COUNTS = {
    "one row": [1],
    "one expert": [300],
    "small": [0, 1, 0, 15, 16, 17, 0],
    "around tiles": [31, 32, 33, 63, 64, 65, 127, 128, 129],
    "large": [0, 255, 256, 257, 513, 2, 0, 0],
    "uneven": [1700, 0, 3, 40, 1],
    "many experts": [(7 * i) % 11 for i in range(75)],
}


def prefix_of(counts, before=0):
    p = [before]
    for c in counts:
        p.append(p[-1] + c)
    return p


def normal(gen, *shape, std=1.0):
    return torch.empty(shape, dtype=BF, device=DEV).normal_(0.0, std, generator=gen)


def rows_with_strangers(gen, prefix, M, cols):
    """[M, cols] bf16; rows of no expert hold infinities and NaN."""
    x = normal(gen, M, cols)
    for sl in (slice(0, prefix[0]), slice(prefix[-1], M)):
        x[sl] = float("nan")
        x[sl, ::3] = float("inf")
    return x


def steps(K):
    return (K / 16 + 16) * 2.0 ** -23


def close(got, want, size, K, half_step):
    """|got - want| <= half_step |want| + the sums' error, with `size` the sums of magnitudes."""
    off = (got.double() - want).abs()
    most = half_step * want.abs() + steps(K) * (1 + half_step) * size
    bad = ~(off <= most)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / most.clamp_min(1e-300)).max()):.2f}"


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (72, 136), (512, 264), (1160, 1048)])
def test_forward_and_gradients(moe, name, K, N):
    counts = COUNTS[name]
    gen = torch.Generator(DEV).manual_seed(len(name) * 1000 + K)
    p = prefix_of(counts, 5)
    M, E = p[-1] + 9, len(counts)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, g, w = rows_with_strangers(gen, p, M, K), rows_with_strangers(gen, p, M, N), normal(gen, E, N, K, std=K ** -0.5)
    status = moe.new_status()
    out, gx = torch.full((M, N), 7.0, dtype=BF, device=DEV), torch.full((M, K), 7.0, dtype=BF, device=DEV)
    assert moe.moe_grouped_linear(x, w, prefix, out=out, status=status) is out
    moe.moe_grouped_linear_grad_x(g, w, prefix, out=gx, status=status)
    gw = moe.moe_grouped_linear_grad_w(g, x, prefix, status=status)
    gw16 = moe.moe_grouped_linear_grad_w(g, x, prefix, dtype=BF, status=status)
    torch.cuda.synchronize()
    moe.check_status(status)
    for t in (out, gx):   # rows of no expert are left as they were
        assert (t[: p[0]] == 7).all() and (t[p[-1]:] == 7).all()
    for e in range(E):
        r = slice(p[e], p[e + 1])
        xe, ge, we = x[r].double(), g[r].double(), w[e].double()
        close(out[r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)
        close(gx[r], ge @ we, ge.abs() @ we.abs(), N, 2.0 ** -8)
        want, size = ge.T @ xe, ge.abs().T @ xe.abs()
        close(gw[e], want, size, max(counts[e], 1), 2.0 ** -24)
        close(gw16[e], want, size, max(counts[e], 1), 2.0 ** -8)


def codes(gen, *shape, dtype=torch.float8_e4m3fn):
    v = torch.empty(shape, device=DEV).normal_(0.0, 100.0, generator=gen).clamp_(-448, 448)
    scales = torch.empty(*shape[:-1], shape[-1] // 128, device=DEV).uniform_(0.25, 4.0, generator=gen) / 100
    return v.to(dtype).view(torch.uint8), scales


def values(c, s):
    return c.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, -1)


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("K,N", [(128, 8), (256, 136), (640, 264), (1152, 1048)])
def test_e4m3(moe, name, K, N):
    counts = COUNTS[name]
    gen = torch.Generator(DEV).manual_seed(len(name) * 1000 + K)
    p = prefix_of(counts, 3)
    M, E = p[-1] + 20, len(counts)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    (x, xs), (w, ws) = codes(gen, M, K), codes(gen, E, N, K)
    for sl in (slice(0, p[0]), slice(p[-1], M)):
        x[sl], xs[sl] = 0x7F, float("nan")
    out = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    status = moe.new_status()
    moe.moe_grouped_linear(x, w, prefix, x_scales=xs, w_scales=ws, out=out, status=status)
    torch.cuda.synchronize()
    moe.check_status(status)
    assert (out[: p[0]] == 7).all() and (out[p[-1]:] == 7).all()
    for e in range(E):
        r = slice(p[e], p[e + 1])
        xe, we = values(x[r], xs[r]), values(w[e], ws[e])
        close(out[r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)


def test_what_a_row_holds_stays_in_it(moe):
    """Infinities and NaN of one row, and of one expert's weights, reach no other row."""
    gen = torch.Generator(DEV).manual_seed(1)
    counts, K, N = [5, 40, 7], 200, 72
    p = prefix_of(counts)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, w = normal(gen, p[-1], K), normal(gen, 3, N, K)
    clean = moe.moe_grouped_linear(x, w, prefix)
    x2 = x.clone()
    x2[7], x2[44, 3] = float("nan"), float("inf")
    got = moe.moe_grouped_linear(x2, w, prefix)
    rest = [r for r in range(p[-1]) if r not in (7, 44)]
    assert torch.equal(got[rest], clean[rest]) and got[7].isnan().all() and not got[44].isfinite().any()
    gw = moe.moe_grouped_linear_grad_w(normal(gen, p[-1], N), x2, prefix)
    assert gw[0].isfinite().all() and gw[2].isfinite().all() and not gw[1].isfinite().all()
    w2 = w.clone()
    w2[1, 5] = float("nan")
    got = moe.moe_grouped_linear(x, w2, prefix)
    assert got[5:45, 5].isnan().all()
    got[5:45, 5] = clean[5:45, 5]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_gradients_add_up(moe, dtype):
    gen = torch.Generator(DEV).manual_seed(2)
    counts, K, N = [0, 70, 1], 136, 72
    p = prefix_of(counts)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, g = normal(gen, p[-1], K), normal(gen, p[-1], N)
    start = torch.randn(3, N, K, device=DEV, generator=gen).to(dtype)
    got = start.clone()
    moe.moe_grouped_linear_grad_w(g, x, prefix, out=got, accumulate=True)
    assert torch.equal(got[0], start[0])
    for e in (1, 2):
        r = slice(p[e], p[e + 1])
        want = g[r].double().T @ x[r].double()
        size = g[r].double().abs().T @ x[r].double().abs()
        # one more sum, rounded
        close(got[e], want + start[e].double(), size + start[e].double().abs(), counts[e],
              2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8)


def test_no_rows(moe):
    prefix = torch.zeros(4, dtype=torch.int32, device=DEV)
    w = torch.ones(3, 16, 24, dtype=BF, device=DEV)
    assert moe.moe_grouped_linear(w.new_empty(0, 24), w, prefix).shape == (0, 16)
    assert moe.moe_grouped_linear_grad_x(w.new_empty(0, 16), w, prefix).shape == (0, 24)
    gw = moe.moe_grouped_linear_grad_w(w.new_empty(0, 16), w.new_empty(0, 24), prefix)
    assert gw.shape == (3, 16, 24) and not gw.any()
    # rows, and none of them an expert's
    x = torch.ones(10, 24, dtype=BF, device=DEV)
    out = torch.full((10, 16), 3.0, dtype=BF, device=DEV)
    moe.moe_grouped_linear(x, w, prefix + 4, out=out)
    gw = moe.moe_grouped_linear_grad_w(out, x, prefix + 4, out=torch.full((3, 16, 24), 5.0, device=DEV))
    assert (out == 3).all() and not gw.any()


@pytest.mark.parametrize("p", [[0, 5, 3, 10], [-2, 4, 6, 8], [0, 4, 30, 40], [12, 4, 4, 8]])
def test_a_bad_prefix_is_cut(moe, p):
    gen = torch.Generator(DEV).manual_seed(3)
    M, K, N = 20, 64, 40
    x, w = normal(gen, M, K), normal(gen, 3, N, K)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    for call in (lambda s: moe.moe_grouped_linear(x, w, prefix, status=s),
                 lambda s: moe.moe_grouped_linear_grad_x(normal(gen, M, N), w, prefix, status=s),
                 lambda s: moe.moe_grouped_linear_grad_w(normal(gen, M, N), x, prefix, status=s)):
        status = moe.new_status()
        call(status)
        with pytest.raises(moe.MoeError) as e:
            moe.check_status(status)
        assert e.value.code == moe.MOE_ERR_BAD_PREFIX


def test_equal_calls_give_equal_bits(moe):
    gen = torch.Generator(DEV).manual_seed(4)
    counts, K, N = [200, 3, 129, 0, 700], 512, 392
    p = prefix_of(counts)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, g, w = normal(gen, p[-1], K), normal(gen, p[-1], N), normal(gen, 5, N, K)
    for call in (lambda: moe.moe_grouped_linear(x, w, prefix), lambda: moe.moe_grouped_linear_grad_x(g, w, prefix),
                 lambda: moe.moe_grouped_linear_grad_w(g, x, prefix)):
        first = call()
        for _ in range(3):
            assert torch.equal(call(), first)
