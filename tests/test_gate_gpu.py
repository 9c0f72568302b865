"""moe_topk_gate and moe_topk_gate_backward against their definitions in 64 bits.

Choices are compared exactly (a choice without bias involves no rounding).
Tolerance of a weight, relative: l - m is one fp32 subtraction, off by
2^-24 |l - m| in the exponent; expf, the division and a sum of E positive
terms by pairs add at most 2 + 1 + log2(E) + E/32 units of 2^-23 (a lane adds its
own E/32 terms one after another). Gradients multiply weights that are that
good with differences g - dot of at most 2 max|g|, so the same tolerance
times 4 max|g| holds in absolute terms, plus the rounding to bf16 (2^-8
relative) where the logits are bf16.
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


def reference(logits, k, score, normalize, scale=1.0):
    """(idx, weights) in 64 bits on the CPU; -inf and NaN are never chosen."""
    l = logits.double().cpu()
    l = torch.where(l.isnan(), -math.inf, l)
    order = torch.sort(l + 0.0, dim=1, descending=True, stable=True).indices[:, :k]
    top = l.gather(1, order)
    on = top > -math.inf
    idx = torch.where(on, order, -1)
    if score == "sigmoid":
        # relative to the largest, so that scores far below zero keep their ratio
        w = torch.nn.functional.logsigmoid(top)
        w = torch.exp(w - w[:, :1]) if normalize else torch.exp(w)
        w = torch.where(on, w, 0)
        w = w / w.sum(1, keepdim=True) if normalize else w
    else:
        d = torch.where(top == top[:, :1], 0.0, top - top[:, :1])
        w = torch.where(on, torch.exp(d), 0)
        full = torch.where(l == top[:, :1], 0.0, l - top[:, :1])
        z = w.sum(1, keepdim=True) if normalize else torch.exp(full).sum(1, keepdim=True)
        w = w / z
    return idx, torch.where(on, w, 0.0) * scale


def rtol(logits):
    l = logits.double()
    l = l[torch.isfinite(l) & (l.abs() < 1e30)]
    spread = float(l.max() - l.min()) if l.numel() else 0.0
    E = logits.shape[1]
    return (min(spread, 110.0) / 2 + 3 + math.log2(E) + E / 32 + 4) * 2.0 ** -23


def make_logits(T, E, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(dtype).cuda()


SHAPES = [(1, 1, 1), (1, 256, 8), (3, 5, 5), (128, 256, 8), (37, 33, 2), (130, 257, 7), (65, 1000, 32), (9, 1024, 6),
          (17, 2048, 8), (5, 2049, 8), (7, 8192, 32), (33, 32, 32)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_matches_definition(moe, T, E, k, dtype, score, normalize):
    l = make_logits(T, E, dtype, T * 7 + E)
    status = moe.new_status()
    idx, w = moe.moe_topk_gate(l, k, score=score, normalize=normalize, scale=2.5, status=status)
    ri, rw = reference(l, k, score, normalize, 2.5)
    assert torch.equal(idx.cpu(), ri)
    torch.testing.assert_close(w.cpu().double(), rw, rtol=rtol(l), atol=1e-30)
    moe.check_status(status)


@pytest.mark.parametrize("E", [64, 256, 300, 2048, 3000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_masks_ties_and_extremes(moe, E, dtype):
    k = 8
    lowest = torch.finfo(dtype).min
    l = make_logits(14, E, torch.float32, 5)
    l[0] = -math.inf                                  # nothing left
    l[1] = -math.inf
    l[1, E - 3] = -2.0                                # one left
    l[2] = lowest                                     # the lowest value is an ordinary logit
    l[3] = lowest
    l[3, 7] = 1.0
    l[4] = 0.25                                       # all equal
    l[5] = torch.where(torch.arange(E) % 2 == 0, 0.0, -0.0)   # signed zeros are equal
    l[6, :5] = math.inf                               # +inf shares the softmax
    l[7, 11] = -math.inf
    l[8] -= 200.0                                     # every sigmoid underflows
    l[9] += 200.0
    l[10] = torch.where(torch.arange(E, device="cuda") < 5, l[10], -math.inf)   # fewer than k
    l[11] = -math.inf
    l[11, 0] = lowest
    l[12] = torch.arange(E, 0, -1)
    l[13] = torch.arange(E) / 4.0
    l = l.to(dtype)
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            status = moe.new_status()
            idx, w = moe.moe_topk_gate(l, k, score=score, normalize=normalize, status=status)
            ri, rw = reference(l, k, score, normalize)
            assert torch.equal(idx.cpu(), ri)
            # fp32 weights below its range come out as 0 or as subnormals
            torch.testing.assert_close(w.cpu().double(), rw, rtol=(110 / 2 + 16 + E / 32) * 2.0 ** -23, atol=2.0 ** -126)
            moe.check_status(status)


def test_gate_nan_is_masked_and_reported(moe):
    l = make_logits(4, 256, torch.float32, 1)
    l[2, 17] = math.nan
    l[3] = math.nan
    for E in (256, 4096):
        ll = torch.nn.functional.pad(l, (0, E - 256), value=-5.0)
        ll[3] = math.nan
        status = moe.new_status()
        idx, w = moe.moe_topk_gate(ll, 8, normalize=False, status=status)
        ri, rw = reference(ll, 8, "softmax", False)
        assert torch.equal(idx.cpu(), ri) and torch.equal(idx[3].cpu(), torch.full((8,), -1))
        torch.testing.assert_close(w.cpu().double(), rw, rtol=rtol(ll[:2]), atol=1e-30)
        assert int(status.item()) == moe.MOE_ERR_BAD_LOGIT


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(64, 256, 8), (9, 40, 4), (6, 4000, 8)])
def test_gate_bias_moves_the_choice_not_the_weights(moe, T, E, k, score, normalize):
    l = make_logits(T, E, torch.float32, 3)
    l[0, :] = -math.inf
    l[0, 2] = 1.0
    bias = (torch.rand(E, generator=torch.Generator().manual_seed(4)) * 0.2).cuda()
    bias[5] = 10.0          # always chosen unless masked
    bias[6] = math.nan      # never chosen
    idx, w = moe.moe_topk_gate(l, k, bias=bias, score=score, normalize=normalize)
    ld, b = l.double().cpu(), bias.double().cpu()
    s = torch.softmax(ld, 1) if score == "softmax" else torch.sigmoid(ld)
    v = torch.where((ld > -math.inf) & ~b.isnan(), s + b, -math.inf)
    idx, w = idx.cpu(), w.cpu().double()
    on = idx >= 0
    assert torch.equal(on.sum(1), (v > -math.inf).sum(1).clamp_max(k))
    got = torch.where(on, v.gather(1, idx.clamp_min(0)), -math.inf)
    want = v.sort(dim=1, descending=True).values[:, :k]
    # a chosen value may be below the one in its place by both sums' rounding
    off = rtol(l) + 2.0 ** -22
    torch.testing.assert_close(torch.where(on, got, 0.0), torch.where(on, want, 0.0), rtol=off, atol=off)
    assert all(len(set(r[r >= 0].tolist())) == int((r >= 0).sum()) for r in idx)
    rw = torch.where(on, s.gather(1, idx.clamp_min(0)), 0.0)
    rw = rw / rw.sum(1, keepdim=True) if normalize else rw
    torch.testing.assert_close(w, rw, rtol=rtol(l), atol=1e-30)


def reference_backward(l, idx, g, score, normalize, scale):
    """The formulas in 64 bits, entry by entry."""
    l, idx, g = l.double().cpu(), idx.cpu(), g.double().cpu() * scale
    out = torch.zeros_like(l)
    for t in range(l.shape[0]):
        on = [(j, int(e)) for j, e in enumerate(idx[t]) if 0 <= e < l.shape[1] and l[t, e] > -math.inf]
        if not on:
            continue
        js, es = [j for j, _ in on], [e for _, e in on]
        top, gt = l[t, es], g[t, js]
        if score == "softmax" and not normalize:
            p = torch.softmax(l[t], 0)
            out[t] = -p * (gt * p[es]).sum()
            for e, gj in zip(es, gt):
                out[t, e] += gj * p[e]
            continue
        if score == "softmax":
            q = torch.softmax(top, 0)
            d = q * (gt - (gt * q).sum())
        else:
            s = torch.sigmoid(top)
            if normalize:
                q = torch.softmax(torch.nn.functional.logsigmoid(top), 0)
                d = q * torch.sigmoid(-top) * (gt - (gt * q).sum())
            else:
                d = gt * s * torch.sigmoid(-top)
        for e, dj in zip(es, d):
            out[t, e] += dj
    return out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (66, 256, 8), (5, 33, 32), (17, 1000, 6), (3, 8192, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_backward_matches_formula(moe, T, E, k, dtype, score, normalize):
    l = make_logits(T, E, dtype, T + E)
    if T > 4 and E > 40:
        l[0] = -math.inf
        l[1] = -math.inf
        l[1, 3] = 0.5
        l[2, 1::2] = -math.inf
        l[3] -= 100.0
    status = moe.new_status()
    idx, _ = moe.moe_topk_gate(l, k, score=score, normalize=normalize)
    if T > 4 and k > 2:
        idx[4, 0] = idx[4, 1]          # one expert twice
        idx[4, 2] = -1
        idx[2, 0] = min(1, E - 1)      # a masked logit named all the same
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(9)).cuda()
    got = moe.moe_topk_gate_backward(l, idx, g, score=score, normalize=normalize, scale=1.5, status=status)
    want = reference_backward(l, idx, g, score, normalize, 1.5)
    assert got.dtype == dtype
    tol = 4 * 1.5 * float(g.abs().max()) * rtol(l)
    torch.testing.assert_close(got.double().cpu(), want, atol=tol, rtol=2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    moe.check_status(status)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gate_backward_matches_differences(moe, score, normalize):
    """Central differences of the forward call: off by step^2 / 6 times a third
    derivative (at most 2 for these scores) and by the forward's rounding over
    the step."""
    T, E, k, step = 5, 24, 4, 2.0 ** -6
    l = make_logits(T, E, torch.float32, 21)
    # logits apart by more than two steps, so that the choice stays
    l = l.argsort(dim=1).argsort(dim=1).float() * 0.125 - 1.5
    idx, _ = moe.moe_topk_gate(l, k, score=score, normalize=normalize)
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(2)).cuda()
    got = moe.moe_topk_gate_backward(l, idx, g, score=score, normalize=normalize).double()
    for e in range(E):
        f = []
        for sign in (1, -1):
            m = l.clone()
            m[:, e] += sign * step
            i2, w = moe.moe_topk_gate(m, k, score=score, normalize=normalize)
            assert torch.equal(i2, idx)
            f.append((w.double() * g.double()).sum(1))
        d = (f[0] - f[1]) / (2 * step)
        total = float(g.abs().sum(1).max())
        torch.testing.assert_close(got[:, e], d, rtol=0, atol=total * (2 * step ** 2 / 6 + rtol(l) / step))


def test_gate_backward_reports_entries_out_of_range(moe):
    l = make_logits(3, 16, torch.float32, 2)
    idx = torch.tensor([[0, 1], [16, 2], [3, -5]], device="cuda")
    g = torch.ones(3, 2, device="cuda")
    status = moe.new_status()
    got = moe.moe_topk_gate_backward(l, idx, g, status=status)
    assert int(status.item()) == moe.MOE_ERR_BAD_TOPK
    torch.testing.assert_close(got.double().cpu(), reference_backward(l, idx, g, "softmax", True, 1.0), rtol=0,
                               atol=8 * rtol(l))


def test_gate_empty_batch_and_side_stream(moe):
    idx, w = moe.moe_topk_gate(torch.empty(0, 16, device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    g = moe.moe_topk_gate_backward(torch.empty(0, 16, device="cuda"), idx, w)
    assert g.shape == (0, 16)
    l = make_logits(300, 256, torch.float32, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = moe.moe_topk_gate(l, 8)
    with torch.cuda.stream(side):
        b = moe.moe_topk_gate(l, 8, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gate_feeds_the_layout(moe):
    import oracle
    l = make_logits(200, 64, torch.bfloat16, 6)
    l[3] = -math.inf
    idx, _ = moe.moe_topk_gate(l, 4)
    lay = moe.moe_get_layout(idx, 64, 8)
    ref = oracle.layout(idx.cpu().numpy(), 64, 8)
    assert (lay.token_dst_row.cpu().numpy() == ref["token_dst_row"]).all()
