"""moe_experts and moe_layer against their definitions in 64 bits.

Tolerance of an output element. With u = 2^-8 the rounding of bf16 and K 2^-24
that of an fp32 sum of K terms against the sum of their magnitudes:
  dg <= H 2^-24 |W_g| |x|, du alike;  silu has slope at most 1.1
  dh <= u |h| + 1.1 dg |up| + |silu| du      (h is held in bf16)
  dout <= u |out| + sum_j |w_j| |w2| (dh + I 2^-24 |h|)
Over all outputs the roundings of h and of out are independent and each is at
most u / sqrt(3) in the mean square, so the error's 2-norm is below
sqrt(2/3) u of the result's; u of it is allowed.
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
    def __init__(self, T, H, I, E, k, e4m3=False, seed=0, masked=0.0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
        self.w13, self.s13, self.w13d = self.weights(g, E, 2 * I, H, e4m3)
        self.w2, self.s2, self.w2d = self.weights(g, E, H, I, e4m3)
        self.idx = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1).indices
        self.w = torch.rand(T, k, device="cuda", generator=g)
        if masked:
            off = torch.rand(T, k, device="cuda", generator=g) < masked
            self.idx[off] = -1
            self.w[off] = math.nan      # what a masked entry weighs does not matter

    @staticmethod
    def weights(g, E, rows, cols, e4m3):
        w = torch.randn(E, rows, cols, device="cuda", generator=g) * cols ** -0.5
        if not e4m3:
            w = w.to(torch.bfloat16)
            return w, None, w.double()
        c = (w * (100 * cols ** 0.5)).clamp(-448, 448).to(torch.float8_e4m3fn)
        s = (torch.rand(E, rows, cols // 128, device="cuda", generator=g) + 0.5) / (100 * cols ** 0.5)
        s[:, 0] = 0.0                   # a row of zero scale
        return c.view(torch.uint8), s, c.double() * s.double().repeat_interleave(128, -1)

    def call(self, moe, **kw):
        return moe.moe_experts(self.x, self.idx, self.w, self.w13, self.w2, w13_scales=self.s13, w2_scales=self.s2, **kw)

    def reference(self):
        """(out, elementwise tolerance) in 64 bits."""
        x, I = self.x.double(), self.I
        out = torch.zeros(self.T, self.H, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        for e in range(self.E):
            t, j = (self.idx == e).nonzero(as_tuple=True)
            if len(t) == 0:
                continue
            y, ya = x[t] @ self.w13d[e].t(), x[t].abs() @ self.w13d[e].abs().t()
            g, up = y[:, :I], y[:, I:]
            s = g * torch.sigmoid(g)
            h = s * up
            d = self.H * EPS * ya
            dh = U * h.abs() + 1.1 * d[:, :I] * up.abs() + s.abs() * d[:, I:] + self.I * EPS * h.abs()
            w = self.w[t, j, None].double()
            out.index_add_(0, t, w * (h @ self.w2d[e].t()))
            tol.index_add_(0, t, w.abs() * (dh @ self.w2d[e].abs().t()))
        return out, tol + U * out.abs() + 1e-30


def check(got, ref, tol, whole=True):
    got = got.double()
    over = (got - ref).abs() - tol
    assert bool((over <= 0).all()), f"worst {float(over.max())} over, at {over.argmax()}"
    if whole and got.numel() >= 4096:    # the mean square needs many outputs
        assert float((got - ref).norm()) <= U * float(ref.norm())


BF16 = [(1, 8, 8, 1, 1), (1, 256, 256, 16, 2), (2, 64, 40, 3, 3), (128, 256, 256, 16, 2), (37, 1160, 520, 24, 3),
        (5, 264, 136, 8, 8), (200, 512, 384, 4, 2), (64, 1024, 128, 3, 1), (300, 136, 72, 2, 2), (1024, 64, 64, 8, 2),
        (16, 7168, 256, 32, 8), (3, 128, 128, 64, 32), (17, 520, 1032, 5, 2), (129, 384, 264, 1, 1)]
E4M3 = [(1, 128, 128, 1, 1), (1, 256, 128, 8, 2), (33, 384, 256, 5, 3), (130, 128, 384, 2, 2), (64, 1024, 512, 32, 8),
        (16, 7168, 256, 16, 4), (257, 256, 128, 3, 1)]
CASES = [(s, False) for s in BF16] + [(s, True) for s in E4M3]


@pytest.mark.parametrize("masked", [0.0, 0.4])
@pytest.mark.parametrize("shape,e4m3", CASES)
def test_experts_match_definition(moe, shape, e4m3, masked):
    p = Problem(*shape, e4m3=e4m3, seed=sum(shape), masked=masked)
    status = moe.new_status()
    got = p.call(moe, status=status)
    check(got, *p.reference())
    moe.check_status(status)


@pytest.mark.parametrize("e4m3", [False, True])
def test_experts_masks_repeats_and_bad_entries(moe, e4m3):
    p = Problem(40, 256, 128, 6, 3, e4m3=e4m3, seed=3)
    p.idx[0] = -1
    p.w[0] = math.inf
    p.idx[1] = 2                        # one expert in every entry
    p.idx[2] = torch.tensor([6, -2, 1])
    p.idx[3] = torch.tensor([1 << 40, -(1 << 40), -1])
    p.idx[4:30, 0] = 5                  # most tokens on one expert
    p.idx[p.idx == 4] = 3               # and nobody on this one
    p.w13[4].view(torch.uint8).fill_(0x7F)   # NaN, in either type (never read)
    p.w[5] = 0.0
    status = moe.new_status()
    got = p.call(moe, status=status)
    p.idx = torch.where((p.idx < 0) | (p.idx >= 6), -1, p.idx)
    ref, tol = p.reference()
    check(got, ref, tol)
    assert bool((got[0] == 0).all()) and bool((got[3] == 0).all())
    assert int(status.item()) == moe.MOE_ERR_BAD_TOPK


@pytest.mark.parametrize("e4m3", [False, True])
def test_experts_every_entry_masked(moe, e4m3):
    p = Problem(9, 256, 128, 4, 2, e4m3=e4m3)
    p.idx.fill_(-1)
    out = torch.full((9, 256), math.nan, dtype=torch.bfloat16, device="cuda")
    p.call(moe, out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("e4m3", [False, True])
def test_experts_tokens_do_not_touch_each_other(moe, e4m3):
    p = Problem(50, 384, 256, 4, 2, e4m3=e4m3, seed=8)
    clean = p.call(moe)
    p.x[7, 11] = math.nan
    p.x[20] = math.inf
    got = p.call(moe)
    keep = [t for t in range(50) if t not in (7, 20)]
    assert torch.equal(got[keep], clean[keep])
    assert bool(got[7].isnan().any()) and not bool(got[20].isfinite().all())


@pytest.mark.parametrize("e4m3", [False, True])
def test_experts_workspace_contents_do_not_matter(moe, e4m3):
    ps = [Problem(60, 384, 256, 12, 3, e4m3=e4m3, seed=s, masked=0.2) for s in (1, 2)]
    n = moe.moe_experts_workspace_size(60, 384, 256, 3, 12)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    first = [p.call(moe, workspace=ws) for p in ps]
    again = [p.call(moe, workspace=ws) for p in ps]
    for p, a, b in zip(ps, first, again):
        check(a, *p.reference())
        assert torch.equal(a, b)


def test_experts_in_a_graph_and_on_a_side_stream(moe):
    p = Problem(24, 512, 256, 8, 2, seed=4)
    want = p.call(moe)
    ws = torch.empty(moe.moe_experts_workspace_size(24, 512, 256, 2, 8), dtype=torch.uint8, device="cuda")
    status, out = moe.new_status(), torch.empty_like(p.x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        p.call(moe, out=out, workspace=ws, status=status, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            p.call(moe, out=out, workspace=ws, status=status)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    moe.check_status(status)


def test_experts_empty_batch(moe):
    p = Problem(4, 64, 64, 2, 1)
    p.x, p.idx, p.w = p.x[:0], p.idx[:0], p.w[:0]
    assert p.call(moe).shape == (0, 64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,e4m3", [(1, 16, 2, False), (130, 40, 4, False), (20, 8, 8, True)])
def test_layer_is_the_gate_and_the_experts(moe, T, E, k, e4m3, dtype):
    p = Problem(T, 256, 128, E, k, e4m3=e4m3, seed=T)
    logits = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dtype)
    logits[0, 1:] = -math.inf
    bias = torch.rand(E, device="cuda")
    for b, score, normalize in ((None, "softmax", True), (bias, "sigmoid", True), (None, "softmax", False)):
        gate = dict(bias=b, score=score, normalize=normalize, scale=1.25)
        p.idx, p.w = moe.moe_topk_gate(logits, k, **gate)
        status = moe.new_status()
        out, idx, w = moe.moe_layer(p.x, logits, k, p.w13, p.w2, w13_scales=p.s13, w2_scales=p.s2, status=status, **gate)
        assert torch.equal(idx, p.idx) and torch.equal(w, p.w)
        assert torch.equal(out, p.call(moe))
        check(out, *p.reference())
        moe.check_status(status)


def test_experts_run_on_dispatched_rows(moe):
    """A rank's share: the dispatch's rows with their localised choices; combined, the ranks' partial rows are the whole."""
    p = Problem(48, 256, 128, 8, 3, seed=6)
    lay = moe.moe_get_layout(p.idx, 8, 2)
    d = moe.moe_dispatch(p.x, p.idx, p.w, 8, 2, lay.token_dst_row, 96)
    lo, mid, hi = lay.rank_prefix.tolist()
    parts = torch.zeros(hi, 256, dtype=torch.bfloat16, device="cuda")
    for r, (a, b) in enumerate(((lo, mid), (mid, hi))):
        parts[a:b] = moe.moe_experts(d.recv_x[a:b], d.recv_topk_idx[a:b], d.recv_topk_weights[a:b],
                                     p.w13[4 * r:4 * r + 4], p.w2[4 * r:4 * r + 4])
    got = moe.moe_combine(parts, lay.token_dst_row).double()
    ref, tol = p.reference()
    # the two ranks' partial rows are rounded to bf16 once more before they are added
    parts_abs = moe.moe_combine(parts.abs(), lay.token_dst_row).double()
    assert bool(((got - ref).abs() <= tol + 2 * U * parts_abs).all())


@pytest.mark.parametrize("T,E,k", [(300, 3, 2), (700, 40, 3), (1024, 1, 1)])
def test_experts_give_the_same_bits_every_time(moe, T, E, k):
    """Groups of many entries, whose sums several CTAs share."""
    p = Problem(T, 512, 384, E, k, seed=T)
    first = p.call(moe)
    for _ in range(5):
        assert torch.equal(p.call(moe), first)
