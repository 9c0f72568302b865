"""moe_adapter_linear against its definition in 64 bits.

Tolerance of an output element: bf16's rounding u = 2^-8 of the result, and
fp32 sums of K and r terms, each off by at most their length times 2^-24 of the
sum of the terms' magnitudes:
  d <= u |out| + (K + r + 4) 2^-24 (|W| |x| + s |B| |A| |x|)
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


class Problem:
    def __init__(self, T, K, N, L, r, spread="rows", seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def bf(*shape, std=1.0):
            return (torch.randn(*shape, device="cuda", generator=g) * std).to(torch.bfloat16)
        self.T, self.K, self.N, self.L, self.r = T, K, N, L, r
        self.x, self.w = bf(T, K), bf(N, K, std=K ** -0.5)
        self.a, self.b = bf(L, r, K, std=K ** -0.5), bf(L, N, r, std=r ** -0.5)
        self.s = torch.rand(L, device="cuda", generator=g) * 2
        idx = torch.randint(-1, L, (T,), device="cuda", generator=g, dtype=torch.int32)
        if spread == "runs":
            idx = idx.sort().values
        if spread == "none":
            idx.fill_(-1)
        if spread == "one":
            idx.fill_(L - 1)
        self.idx = idx

    def call(self, moe, **kw):
        return moe.moe_adapter_linear(self.x, self.w, self.idx, self.a, self.b, self.s, **kw)

    def reference(self):
        x = self.x.double()
        y, m = x @ self.w.double().t(), x.abs() @ self.w.double().abs().t()
        for i in range(self.L):
            t = (self.idx == i).nonzero()[:, 0]
            a, b, s = self.a[i].double(), self.b[i].double(), self.s[i].double()
            y[t] += s * (x[t] @ a.t()) @ b.t()
            m[t] += s * (x[t].abs() @ a.abs().t()) @ b.abs().t()
        return y, U * y.abs() + (self.K + self.r + 4) * EPS * m + 1e-30


def check(got, ref, tol):
    over = (got.double() - ref).abs() - tol
    assert bool((over <= 0).all()), f"worst {float(over.max())} over, at {over.argmax()}"


SHAPES = [(1, 8, 8, 1, 8), (1, 7168, 256, 4, 16), (2, 64, 72, 2, 128), (128, 512, 1000, 48, 16), (317, 1048, 1336, 7, 24),
          (300, 256, 520, 3, 128), (1000, 512, 384, 16, 64), (16, 2048, 136, 2, 72), (65, 72, 200, 5, 40),
          (129, 264, 264, 300, 8), (2500, 128, 768, 9, 32), (33, 4096, 4096, 3, 16)]


@pytest.mark.parametrize("spread", ["rows", "runs", "none", "one"])
@pytest.mark.parametrize("shape", SHAPES)
def test_adapter_matches_definition(moe, shape, spread):
    p = Problem(*shape, spread=spread, seed=sum(shape))
    status = moe.new_status()
    check(p.call(moe, status=status), *p.reference())
    moe.check_status(status)


@pytest.mark.parametrize("T", [3, 40, 300])
def test_adapter_reaches_only_its_rows(moe, T):
    p = Problem(T, 264, 392, 4, 16, seed=T)
    p.idx[0], p.idx[1], p.idx[2] = 2, -1, 1
    clean = p.call(moe)
    p.a[2, 3, 5] = math.nan
    p.b[2, 7] = math.inf
    got = p.call(moe)
    others = p.idx != 2
    assert torch.equal(got[others], clean[others])
    assert bool(got[0].isnan().any())


def test_adapter_rows_do_not_touch_each_other(moe):
    p = Problem(70, 264, 392, 4, 16, seed=5)
    clean = p.call(moe)
    p.x[9, 1] = math.nan
    p.x[33] = math.inf
    got = p.call(moe)
    keep = [t for t in range(70) if t not in (9, 33)]
    assert torch.equal(got[keep], clean[keep]) and bool(got[9].isnan().all())


def test_adapter_reports_an_index_out_of_range(moe):
    p = Problem(20, 64, 64, 3, 8, seed=1)
    p.idx[4], p.idx[5] = 3, -2
    status = moe.new_status()
    got = p.call(moe, status=status)
    check(got, *p.reference())          # the reference gives such rows no adapter either
    assert int(status.item()) == moe.MOE_ERR_BAD_ADAPTER


def test_adapter_zero_rank_tail_is_a_lower_rank(moe):
    p, q = Problem(50, 128, 128, 3, 32, seed=2), Problem(50, 128, 128, 3, 16, seed=2)
    p.a[:, 16:], p.b[:, :, 16:] = 0, 0
    q.x, q.w, q.s, q.idx = p.x, p.w, p.s, p.idx
    q.a, q.b = p.a[:, :16].contiguous(), p.b[:, :, :16].contiguous()
    check(p.call(moe), *q.reference())


def test_adapter_workspace_graph_and_side_stream(moe):
    ps = [Problem(60, 520, 640, 6, 24, seed=s) for s in (1, 2)]
    ws = torch.full((moe.moe_adapter_linear_workspace_size(60, 520, 640, 6, 24),), 0xFF, dtype=torch.uint8, device="cuda")
    first = [p.call(moe, workspace=ws) for p in ps]
    again = [p.call(moe, workspace=ws) for p in ps]
    for p, a, b in zip(ps, first, again):
        check(a, *p.reference())
        assert torch.equal(a, b)
    status, out = moe.new_status(), torch.empty_like(first[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        ps[0].call(moe, out=out, workspace=ws, status=status, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, first[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            ps[1].call(moe, out=out, workspace=ws, status=status)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[1])
    moe.check_status(status)


def test_adapter_empty_batch(moe):
    p = Problem(4, 64, 64, 2, 8)
    p.x, p.idx = p.x[:0], p.idx[:0]
    assert p.call(moe).shape == (0, 64)


def test_adapter_gives_the_same_bits_every_time(moe):
    p = Problem(1500, 512, 384, 6, 64, seed=3)
    first = p.call(moe)
    for _ in range(5):
        assert torch.equal(p.call(moe), first)


# Sorted by adapter: tiles of 128 and of 256 rows that several adapters share, ranks of
# one and two blocks, more adapters than rows to a tile, tiles that CTAs share.
TILED = [(4100, 264, 4104, 5, 64), (4100, 264, 4104, 40, 72), (5000, 64, 2056, 9, 128), (6000, 128, 4096, 200, 128),
         (513, 1288, 1288, 2, 128), (20000, 64, 4096, 1000, 8), (1030, 2056, 1032, 30, 104), (2000, 8, 4096, 2, 128),
         (600, 8200, 1064, 2, 128), (1100, 8328, 5000, 3, 64)]


@pytest.mark.parametrize("spread", ["rows", "runs", "none", "one"])
@pytest.mark.parametrize("shape", TILED)
def test_adapter_tiles_match_definition(moe, shape, spread):
    p = Problem(*shape, spread=spread, seed=sum(shape))
    status = moe.new_status()
    need = moe.moe_adapter_linear_workspace_size(*shape)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    first = p.call(moe, workspace=ws[:need], status=status)
    check(first, *p.reference())
    assert torch.equal(p.call(moe, workspace=ws[:need], status=status), first)
    assert bool((ws[need:] == 0xFF).all())
    moe.check_status(status)


@pytest.mark.parametrize("shape", [(4100, 264, 4104, 5, 64), (1030, 2056, 1032, 30, 104)])
def test_adapter_in_a_tile_reaches_only_its_rows(moe, shape):
    p = Problem(*shape, seed=7)
    clean = p.call(moe)
    p.a[2, 3, 5] = math.nan
    p.b[2, 7] = math.inf
    p.x[9, 1] = math.nan
    p.x[33] = math.inf
    got = p.call(moe)
    keep = p.idx != 2
    hit = p.idx == 2
    keep[9] = keep[33] = False
    assert torch.equal(got[keep], clean[keep])
    assert bool(got[hit].isnan().all()) and bool(got[9].isnan().all())


def test_adapter_tiles_report_an_index_out_of_range(moe):
    p = Problem(4100, 264, 4104, 5, 64, seed=1)
    p.idx[4], p.idx[5] = 5, -2
    status = moe.new_status()
    check(p.call(moe, status=status), *p.reference())
    assert int(status.item()) == moe.MOE_ERR_BAD_ADAPTER
