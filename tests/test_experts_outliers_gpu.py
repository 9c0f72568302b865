"""E4M3 experts where one channel of x, or of h, is thousands of times the others.

The weights of the large channel are zero, so that outputs come from the others alone, at the accuracy that they
have without it. Tolerance: the roundings of h (eight bits) and out are independent and at most u / sqrt(3) in the
mean square, u = 2^-8, together sqrt(2/3) u. An element of a block whose largest is M is held to 2^-22 M where it
is below 2^-14 M, else exactly (x) or to eight bits (h). With M = 2^13 and others of about 1 that is an error of 2^-9
for elements below 1/4, in the mean square 2^-9 sqrt(0.6) if six tenths are; through both of h's factors at
most 1.8 times that, 0.0027: with 0.0032 from above, 0.0042, which is below 1.1 u.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


def weights(g, E, rows, cols):
    codes = (torch.randn(E, rows, cols, device="cuda", generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = (torch.rand(E, rows, cols // 128, device="cuda", generator=g) + 0.5) / (100 * cols ** 0.5)
    return codes.view(torch.uint8), scales


def exact(x, idx, w, w13, s13, w2, s2):
    def wide(codes, scales):
        return codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, -1)
    w13, w2, I = wide(w13, s13), wide(w2, s2), w2.shape[2]
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(w13.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        y = x[t].double() @ w13[e].t()
        h = torch.nn.functional.silu(y[:, :I]) * y[:, I:]
        out.index_add_(0, t, w[t, j, None].double() * (h @ w2[e].t()))
    return out


# a block is scaled so that its largest is in [128, 256): both ends of that
@pytest.mark.parametrize("large", [2.0 ** 12, 2.0 ** 13 - 2.0 ** 5])
@pytest.mark.parametrize("where", ["x", "h"])
@pytest.mark.parametrize("T,H,I,E,k", [(40, 384, 128, 4, 2), (300, 256, 256, 3, 2)])
def test_outliers_cost_the_others_no_bits(moe, T, H, I, E, k, where, large):
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    (w13, s13), (w2, s2) = weights(g, E, 2 * I, H), weights(g, E, H, I)
    if where == "x":
        x[:, 5::128] = large
        w13[:, :, 5::128] = 0
    else:
        w13[:, 5:I:128, 1:] = 0                     # h[5] = silu(x[0] of about 1) times large ones
        w13[:, I + 5::128, 1:] = 0
        x[:, 0] = 1.0
        one = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
        w13[:, 5:I:128, 0] = w13[:, I + 5::128, 0] = one
        s13[:, 5:I:128], s13[:, I + 5::128] = 1.0, large
        w2[:, :, 5::128] = 0
    idx = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1).indices
    w = torch.rand(T, k, device="cuda", generator=g)
    status = moe.new_status()
    got = moe.moe_experts(x, idx, w, w13, w2, w13_scales=s13, w2_scales=s2, status=status).double()
    want = exact(x, idx, w, w13, s13, w2, s2)
    moe.check_status(status)
    assert float((got - want).norm()) <= 1.1 * U * float(want.norm())


# both ends of what a block's largest is scaled to
@pytest.mark.parametrize("largest", [128.0, 255.0])
def test_small_elements_beside_a_large_one(moe, largest):
    """Element t of token t comes out alone, times 64: silu(64) = 64 in fp32, an up row and a row of w2 of a single
    one each, so h and out are a power of two times it, exactly. Elements down to 2^-7, 2^-14 of 128, are
    exact in x with eight bits; smaller ones are off by 2^-15 at most, 2^-22 of 128, and what is kept of them, a multiple
    of 2^-14 below 2^-7, has fewer than eight bits."""
    T = 126
    x = torch.zeros(T, 128, dtype=torch.float64)
    for t in range(T):
        x[t, 0], x[t, 1] = 64.0, largest
        x[t, 2 + t] = (1.0 + (t * 37 % 128) / 128) * 2.0 ** (6 - t % 20)      # [2^-13, 128)
    x = x.cuda()
    one = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
    w13, w2 = (torch.zeros(1, n, 128, dtype=torch.uint8, device="cuda") for n in (256, 128))
    own = torch.arange(2, 128)
    w13[0, :128, 0] = one
    w13[0, 128 + own, own] = one
    w2[0, own, own] = one
    got = moe.moe_experts(x.bfloat16(), torch.zeros(T, 1, dtype=torch.int64, device="cuda"), torch.ones(T, 1, device="cuda"),
                          w13, w2, w13_scales=torch.ones(1, 256, 1, device="cuda"),
                          w2_scales=torch.ones(1, 128, 1, device="cuda")).double()
    want = 64 * x
    want[:, :2] = 0
    small = want < 64 * 2.0 ** -7
    assert torch.equal(got[~small], want[~small])
    assert bool(((got - want)[small].abs() <= 64 * 2.0 ** -15).all())
