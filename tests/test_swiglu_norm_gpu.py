"""moe_swiglu, moe_add_rms_norm and their gradients against their formulas in 64 bits.

Tolerances. A rounding to bf16 is off by 2^-8 of the value at most, one to fp32 by 2^-24. The sigmoid's exp and quotient
are the fast ones: exp2 of a rounded product, off by 2^-22 + |z| 2^-23 for |z| up to 88, and a quotient off by 2^-22: with
the handful of products around it under 2^-16 for all z that the tests have (|z| < 30)."""
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


def normal(gen, *shape, std=1.0):
    return torch.empty(shape, dtype=BF, device=DEV).normal_(0.0, std, generator=gen)


def close(got, want, rel, floor=0.0):
    off, most = (got.double() - want).abs(), rel * want.abs() + floor
    bad = ~(off <= most)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / (most + 1e-300)).max()):.2f}"


def check_codes(codes, scales, want, rel):
    """Codes and scales of rows `want` that the kernel has within `rel`: scales to `rel` and a rounding, codes off the
    quotient by half a step (2^-4 of it, or of the smallest normal 2^-6) and what `rel` moves it."""
    blocks = want.unflatten(-1, (-1, 128))
    s = blocks.abs().amax(-1) / 448
    close(scales, s, rel + 2.0 ** -23)
    q = torch.where(s[..., None] > 0, blocks / s[..., None], 0.0).flatten(-2)
    got = codes.view(torch.float8_e4m3fn).double()
    assert not got.isnan().any()
    close(got, q, 2.0 ** -4 + 4 * rel, 2.0 ** -10)


FAST = 2.0 ** -16


@pytest.mark.parametrize("M,I,rows", [(1, 8, None), (1, 128, 1), (7, 264, 5), (300, 1416, 299), (33, 2048, 0), (5, 4096, None),
                                      (2000, 384, 1024)])
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu(moe, M, I, rows, weighted):
    gen = torch.Generator(DEV).manual_seed(M + I)
    n = M if rows is None else rows
    gu, g = normal(gen, M, 2 * I, std=3.0), normal(gen, M, I)
    gu[n:], g[n:] = float("nan"), float("nan")
    w = torch.randn(M, device=DEV, generator=gen) if weighted else None
    num = None if rows is None else torch.tensor([rows], dtype=torch.int32, device=DEV)
    keep = dict(row_weights=w, num_rows=num, status=moe.new_status())
    out = torch.full((M, I), 7.0, dtype=BF, device=DEV)
    moe.moe_swiglu(gu, out=out, **keep)
    dgu = torch.full((M, 2 * I), 7.0, dtype=BF, device=DEV)
    dw = torch.full((M,), 7.0, device=DEV) if weighted else None
    got = moe.moe_swiglu_backward(gu, g, out=dgu, grad_row_weights=dw, **keep)
    assert got[0] is dgu or torch.equal(got[0], dgu)
    moe.check_status(keep["status"])
    assert (out[n:] == 7).all() and (dgu[n:] == 7).all() and (dw is None or (dw[n:] == 7).all())
    gu64 = gu[:n].double().requires_grad_()
    w64 = (w[:n] if weighted else torch.ones(n, device=DEV)).double().requires_grad_()
    gate, up = gu64.chunk(2, 1)
    y = torch.nn.functional.silu(gate) * up * w64[:, None]
    close(out[:n], y.detach(), 2.0 ** -8 + FAST)
    want, want_w = torch.autograd.grad(y, (gu64, w64), g[:n].double())
    # 1 + g (1 - s) may cancel near g = -1.28: its terms are of size 1, off by FAST each
    sig = torch.sigmoid(gate.detach())
    floor = torch.cat([(g[:n].double() * w64.detach()[:, None] * up.detach() * sig).abs() * 4 * FAST, torch.zeros_like(sig)], 1)
    close(dgu[:n], want, 2.0 ** -8 + FAST, floor)
    if weighted:
        size = (g[:n].double() * torch.nn.functional.silu(gate.detach()) * up.detach()).abs().sum(1)
        close(dw[:n], want_w, 0, (FAST + (I / 32 + 8) * 2.0 ** -24) * size)
    if I % 128 == 0:
        codes = torch.full((M, I), 9, dtype=torch.uint8, device=DEV)
        scales = torch.full((M, I // 128), 9.0, device=DEV)
        moe.moe_swiglu(gu, quantize_fp8=True, out=codes, out_scales=scales, **keep)
        assert (codes[n:] == 9).all() and (scales[n:] == 9).all()
        check_codes(codes[:n], scales[:n], y.detach(), FAST)


def test_swiglu_gradient_against_differences(moe):
    gen = torch.Generator(DEV).manual_seed(5)
    M, I = 3, 16
    gu, g = normal(gen, M, 2 * I), normal(gen, M, I)
    w = torch.rand(M, device=DEV, generator=gen)
    dgu, dw = moe.moe_swiglu_backward(gu, g, row_weights=w)

    def loss(gu, w):
        gate, up = gu.double().chunk(2, 1)
        return (torch.nn.functional.silu(gate) * up * w.double()[:, None] * g.double()).sum()

    step = 2.0 ** -12   # central differences: off by step^2 times a third derivative (under 8 here) over 6
    for r, c in [(0, 0), (1, 5), (2, 17), (0, 31)]:
        d = torch.zeros(M, 2 * I, dtype=torch.float64, device=DEV)
        d[r, c] = step
        want = (loss(gu.double() + d, w) - loss(gu.double() - d, w)) / (2 * step)
        assert abs(float(dgu[r, c]) - float(want)) <= (2.0 ** -8 + FAST) * abs(float(want)) + 1e-6
    for r in range(M):
        d = torch.zeros(M, dtype=torch.float64, device=DEV)
        d[r] = step
        want = (loss(gu, w.double() + d) - loss(gu, w.double() - d)) / (2 * step)
        assert abs(float(dw[r]) - float(want)) <= 1e-4 * max(1.0, abs(float(want)))


def test_swiglu_far_gates(moe):
    """Where exp overflows or vanishes, and rows without a size."""
    gate = torch.tensor([-3e38, -1e4, -100.0, -89.0, -88.0, 0.0, 88.0, 3e38], device=DEV).to(BF)
    gu = torch.cat([gate.repeat(16), torch.ones(128, dtype=BF, device=DEV)])[None].contiguous()
    out, _ = moe.moe_swiglu(gu)
    want = torch.nn.functional.silu(gate.double()).repeat(16)
    close(out[0], want, 2.0 ** -8 + FAST, 1e-35)   # products of e^-88 lie near the smallest normal
    dgu, _ = moe.moe_swiglu_backward(gu, torch.ones(1, 128, dtype=BF, device=DEV))
    assert dgu.isfinite().all()
    zero = torch.zeros(2, 512, dtype=BF, device=DEV)
    codes, scales = moe.moe_swiglu(zero, quantize_fp8=True)
    assert not codes.any() and not scales.any()


@pytest.mark.parametrize("bad", [-1, 6])
def test_swiglu_row_number_out_of_range(moe, bad):
    gu = torch.ones(5, 32, dtype=BF, device=DEV)
    num = torch.tensor([bad], dtype=torch.int32, device=DEV)
    status = moe.new_status()
    moe.moe_swiglu(gu, num_rows=num, status=status)
    with pytest.raises(moe.MoeError) as e:
        moe.check_status(status)
    assert e.value.code == moe.MOE_ERR_CAPACITY


SIZES = [(1, 8), (1, 128), (3, 264), (9, 1024), (130, 1416), (700, 4096), (5, 4104), (128, 7168), (17, 8192), (4, 8200),
         (2500, 136), (3, 16256), (333, 16384)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_norm(moe, T, H, with_residual, wide):
    gen = torch.Generator(DEV).manual_seed(T + H)
    x, w = normal(gen, T, H), (1 + 0.3 * torch.randn(H, device=DEV, generator=gen))
    w = w if wide else w.to(BF)
    res = normal(gen, T, H, std=3.0) if with_residual else None
    quantize = H % 128 == 0
    status = moe.new_status()
    r = moe.moe_add_rms_norm(x, w, residual=res, eps=1e-5, quantize_fp8=quantize, status=status)
    h = x.double() + (res.double() if with_residual else 0)
    y = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    # H squares and a dozen roundings: the sum's relative error is that of positive terms, a lane's share of them in turn
    rel = (H / 256 + 32) * 2.0 ** -24
    close(r.out, y, 2.0 ** -8 + rel, 0)
    if with_residual:   # a sum of two bf16 in fp32, rounded once more
        close(r.residual, h, 2.0 ** -8 + 2.0 ** -23)
    else:
        assert r.residual is None
    if quantize:
        check_codes(r.codes, r.scales, y, rel)
        only = moe.moe_add_rms_norm(x, w, residual=res, eps=1e-5, quantize_fp8=True, bf16_out=False)
        assert only.out is None and torch.equal(only.codes, r.codes) and torch.equal(only.scales, r.scales)
    else:
        assert r.codes is None and r.scales is None

    kept = r.residual if with_residual else x
    g, gr = normal(gen, T, H), normal(gen, T, H) if with_residual else None
    gx, gw = moe.moe_add_rms_norm_backward(kept, w, g, grad_residual=gr, eps=1e-5, status=status)
    moe.check_status(status)
    k64, w64 = kept.double().requires_grad_(), w.double().requires_grad_()
    inv = 1 / (k64.square().mean(1, keepdim=True) + 1e-5).sqrt()
    wx, ww = torch.autograd.grad(k64 * inv * w64, (k64, w64), g.double())
    if with_residual:
        wx = wx + gr.double()
    n, inv = (k64 * inv).detach(), inv.detach()
    d = (g.double() * w64).detach()
    # terms that may cancel
    size = inv * (d.abs() + n.abs() * (d * n).abs().mean(1, keepdim=True)) + (gr.double().abs() if with_residual else 0)
    close(gx, wx, 2.0 ** -8, (rel + 2.0 ** -20) * size)
    close(gw, ww, 0, (rel + (T + 8) * 2.0 ** -24) * (g.double() * n).abs().sum(0))


def test_norm_in_place(moe):
    gen = torch.Generator(DEV).manual_seed(6)
    x, res, w = normal(gen, 40, 1024), normal(gen, 40, 1024), normal(gen, 1024)
    want = moe.moe_add_rms_norm(x, w, residual=res)
    kept = res.clone()
    got = moe.moe_add_rms_norm(x, w, residual=kept, residual_out=kept)
    assert torch.equal(got.out, want.out) and torch.equal(kept, want.residual)
    g = normal(gen, 40, 1024)
    gx, gw = moe.moe_add_rms_norm_backward(kept, w, g)
    g2 = g.clone()
    gx2, gw2 = moe.moe_add_rms_norm_backward(kept, w, g2, out=g2)
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)


def test_norm_of_zeros_and_rows_that_are_not_finite(moe):
    x = torch.zeros(4, 256, dtype=BF, device=DEV)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    x[3] = 1.0
    r = moe.moe_add_rms_norm(x, torch.ones(256, device=DEV), quantize_fp8=True)
    assert not r.out[0].any() and not r.codes[0].any() and not r.scales[0].any()
    assert r.out[1].isnan().all() and r.out[2, 200].isnan() and torch.allclose(r.out[3].float(), torch.ones(256, device=DEV))


def test_norm_codes_are_the_dispatchs(moe):
    """The rows that the norm quantises go through moe_dispatch as they are."""
    gen = torch.Generator(DEV).manual_seed(7)
    T, H, E, R = 64, 512, 16, 4
    r = moe.moe_add_rms_norm(normal(gen, T, H), torch.ones(H, device=DEV), quantize_fp8=True)
    idx = torch.rand(T, E, device=DEV, generator=gen).topk(2, 1).indices
    lay = moe.moe_get_layout(idx, E, R)
    d = moe.moe_dispatch(r.codes, idx, None, E, R, lay.token_dst_row, T * 2, x_scales=r.scales)
    n = int(lay.rank_prefix[-1])
    src = d.recv_src_idx[:n].long()
    assert torch.equal(d.recv_x[:n], r.codes[src]) and torch.equal(d.recv_x_scales[:n], r.scales[src])


@pytest.mark.parametrize("T,H", [(1, 64), (1000, 256)])
def test_norm_backward_without_rows_and_twice(moe, T, H):
    gen = torch.Generator(DEV).manual_seed(8)
    x, w, g = normal(gen, T, H), normal(gen, H), normal(gen, T, H)
    a, b = moe.moe_add_rms_norm_backward(x, w, g), moe.moe_add_rms_norm_backward(x, w, g)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    gx, gw = moe.moe_add_rms_norm_backward(x[:0], w, g[:0])
    assert gx.shape == (0, H) and not gw.any()


def test_offsets_beyond_32_bits(moe):
    """2.3 * 10^9 elements; the last rows."""
    gen = torch.Generator(DEV).manual_seed(13)
    M, I = 280_000, 4096
    gu = torch.zeros(M, 2 * I, dtype=BF, device=DEV)
    gu[-3:] = normal(gen, 3, 2 * I)
    want = torch.nn.functional.silu(gu[-3:, :I].double()) * gu[-3:, I:].double()
    out, _ = moe.moe_swiglu(gu)
    close(out[-3:], want, 2.0 ** -8 + FAST)
    c, s = moe.moe_swiglu(gu, quantize_fp8=True)
    check_codes(c[-3:], s[-3:], want, FAST)
    grad = torch.zeros(M, I, dtype=BF, device=DEV)
    grad[-3:] = normal(gen, 3, I)
    d, _ = moe.moe_swiglu_backward(gu, grad)
    few, _ = moe.moe_swiglu_backward(gu[-3:].contiguous(), grad[-3:].contiguous())
    assert torch.equal(d[-3:], few) and not d[0].any()
    del out, c, s, grad, d
    w = normal(gen, 2 * I)
    r = moe.moe_add_rms_norm(gu, w, residual=gu)
    few = moe.moe_add_rms_norm(gu[-3:].contiguous(), w, residual=gu[-3:].contiguous())
    assert torch.equal(r.out[-3:], few.out) and torch.equal(r.residual[-3:], few.residual)
    gx, gw = moe.moe_add_rms_norm_backward(gu, w, r.out, eps=1.0)
    few = moe.moe_add_rms_norm_backward(gu[-3:].contiguous(), w, r.out[-3:].contiguous(), eps=1.0)
    assert torch.equal(gx[-3:], few[0])
    close(gw, few[1].double(), 2.0 ** -20, 2.0 ** -20 * float(few[1].abs().max()))   # three rows in another order


def test_a_limit_alone_changes_nothing_for_the_norms_gradient(moe):
    gen = torch.Generator(DEV).manual_seed(14)
    x, w, g = normal(gen, 500, 1024), normal(gen, 1024), normal(gen, 500, 1024)
    want, status = moe.moe_add_rms_norm_backward(x, w, g), moe.new_status()
    with moe.test_wait_limits(20_000_000):
        got = moe.moe_add_rms_norm_backward(x, w, g, status=status)
    moe.check_status(status)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_in_a_graph_and_on_another_stream(moe):
    gen = torch.Generator(DEV).manual_seed(15)
    M, H = 60, 512
    x, res, w, g, gu = normal(gen, M, H), normal(gen, M, H), normal(gen, H), normal(gen, M, H), normal(gen, M, 2 * H)
    rw, num = torch.rand(M, device=DEV, generator=gen), torch.tensor([M], dtype=torch.int32, device=DEV)
    ws = torch.empty(moe.moe_add_rms_norm_backward_workspace_size(M, H), dtype=torch.uint8, device=DEV)
    status = moe.new_status()

    def step(**kw):
        kw["status"] = status
        n = moe.moe_add_rms_norm(x, w, residual=res, quantize_fp8=True, **kw)
        b = moe.moe_add_rms_norm_backward(n.residual, w, g, grad_residual=g, workspace=ws, **kw)
        h, _ = moe.moe_swiglu(gu, row_weights=rw, num_rows=num, **kw)
        q = moe.moe_swiglu(gu, row_weights=rw, num_rows=num, quantize_fp8=True, **kw)
        d = moe.moe_swiglu_backward(gu, g, row_weights=rw, num_rows=num, **kw)
        return [n.out, n.residual, n.codes, n.scales, *b, h, *q, *d]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    segments = [s for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream]
    for t in got:   # outputs are memory of the stream that wrote them
        assert any(s["address"] <= t.data_ptr() < s["address"] + s["total_size"] for s in segments)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    num.fill_(7)   # the number of rows stays on the device
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[6][:7], want[6][:7]) and not outs[6][7:].any()
    moe.check_status(status)
