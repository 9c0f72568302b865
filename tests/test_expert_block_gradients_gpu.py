"""The expert block's gradients of its output alone, without the residual's share, path by path.

The reference is in 64 bits on the CPU with a rounding to bf16 wherever the block rounds, forward and backward, so that what
is left are values that fall to the other side of a rounding: few, by 2^-8 of themselves each. The tolerance of 2^-7 of a
gradient's norm covers two whole roundings of every value."""
from __future__ import annotations

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOLERANCE = 2.0 ** -7
NAMES = ("x", "norm", "router", "w13", "w2")


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, ROOT)
    from examples import expert_block
    return expert_block


def bf16(t):
    return t.to(torch.bfloat16).to(t.dtype)


class Rounded(torch.autograd.Function):
    """A value and its gradient, each rounded to bf16."""

    @staticmethod
    def forward(ctx, t):
        return bf16(t)

    @staticmethod
    def backward(ctx, grad):
        return bf16(grad)


class GradientRounded(torch.autograd.Function):
    @staticmethod
    def forward(ctx, t):
        return t.clone()

    @staticmethod
    def backward(ctx, grad):
        return bf16(grad)


def reference(block, x, residual, idx, target, without=None):
    """Gradients of sum(out * target), on the CPU; `without` leaves a path out: "router" or "rows"."""
    wide = [t.detach().cpu().double().requires_grad_() for t in (x, *block.parameters())]
    x, norm, router, w13, w2 = wide
    residual, idx, target = residual.cpu().double(), idx.cpu(), target.cpu().double()

    def normed(h):
        return h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * norm

    # the norm takes h as it is, its gradient h as it was kept
    h = x + residual
    kept = GradientRounded.apply(h + (bf16(h) - h).detach())
    n = normed(kept)
    n = Rounded.apply(n + (normed(h) - n).detach())
    to_router, to_rows = GradientRounded.apply(n), GradientRounded.apply(n)
    if without == "router":
        to_router = to_router.detach()
    if without == "rows":
        to_rows = to_rows.detach()
    logits = Rounded.apply(to_router @ router.T)
    weights = torch.softmax(logits.gather(1, idx), 1)
    if without == "router":
        weights = weights + 0 * router.sum()   # a gradient of zeros
    out = torch.zeros_like(n)
    for e in range(block.num_experts):
        t, j = (idx == e).nonzero(as_tuple=True)
        rows = GradientRounded.apply(to_rows[t])
        gate, up = Rounded.apply(rows @ w13[e].T).chunk(2, 1)
        act = Rounded.apply(torch.nn.functional.silu(gate) * up * weights[t, j, None])
        out = out.index_add(0, t, Rounded.apply(act @ w2[e].T))
    return [bf16(g) for g in torch.autograd.grad(Rounded.apply(out), wide, target)]


def gradients(ex, block, x, residual, target):
    """(idx, gradients of sum(out * target)) by the example's functions."""
    s = block.status
    x, (norm, router, w13, w2) = x.detach().requires_grad_(), [p.detach().requires_grad_() for p in block.parameters()]
    n, _ = ex.AddRmsNorm.apply(x, residual, norm, s)
    idx, topk_weights = ex.TopkGate.apply(n @ router.T, block.num_topk, block.options, s)
    to = ex.Routing(idx, block.num_experts, s)
    h = ex.Swiglu.apply(ex.GroupedLinear.apply(ex.Dispatch.apply(n, to), w13, to.prefix, s), to.weights(topk_weights), s)
    out = ex.Combine.apply(ex.GroupedLinear.apply(h, w2, to.prefix, s), to)
    return idx, torch.autograd.grad(out, [x, norm, router, w13, w2], target)


def off(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (300, 256, 128, 8, 2), (77, 512, 384, 16, 4)])
def test_gradients_of_the_output(ex, T, H, I, E, k):
    block = ex.Block(H, I, E, k)
    gen = torch.Generator("cuda").manual_seed(41)
    x, residual, target = (torch.randn(T, H, generator=gen, device="cuda").bfloat16() for _ in range(3))
    idx, got = gradients(ex, block, x, residual, target)
    ex.moe.check_status(block.status)
    want = reference(block, x, residual, idx, target)
    for name, a, b in zip(NAMES, got, want):
        assert off(a, b) < TOLERANCE, name
    # a path that is missing shows
    for without, seen in (("router", ("x", "norm")), ("rows", ("x", "norm"))):
        other = reference(block, x, residual, idx, target, without)
        for name, a, b in zip(NAMES, other, want):
            assert name not in seen or off(a, b) > 4 * TOLERANCE, (without, name)
