"""The operators around a dispatch as they are used together: the expert block's steps against their definitions in 64
bits, in a CUDA graph, and its gradients.

Tolerances, relative to a result's norm. A rounding to bf16 is off by at most 2^-8 of the value; the roundings that one
result goes through on its way (norm, product, activation, product, combine; backward about as many again) add up to no
more than their number times that where the steps between them do not amplify, which random weights of unit gain do not
beyond a factor of two. E4M3 rows and activations are off by 2^-4 of each element at most, 2^-4 / sqrt(3) of the norm."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, ROOT)
    from examples import expert_block
    return expert_block


def inputs(T, H, seed=1):
    gen = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(T, H, generator=gen, device="cuda").bfloat16() for _ in range(2)]


def reference(block, x, residual, idx, w13, w2, params=None):
    """(out, kept) in 64 bits for the given choice."""
    norm, router = params[:2] if params else (block.norm.double(), block.router.double())
    kept = x.double() + residual.double()
    n = kept / (kept.square().mean(1, keepdim=True) + 1e-6).sqrt() * norm
    weights = torch.softmax((n @ router.T).gather(1, idx), 1)
    out = torch.zeros_like(n)
    for e in range(block.num_experts):
        t, j = (idx == e).nonzero(as_tuple=True)
        gate, up = (n[t] @ w13[e].T).chunk(2, 1)
        h = torch.nn.functional.silu(gate) * up * weights[t, j, None]
        out = out.index_add(0, t, h @ w2[e].T)
    return out, kept


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("T", [1, 37, 600])
@pytest.mark.parametrize("e4m3", [False, True])
def test_step(ex, T, e4m3):
    block = ex.Block(512, 256, 16, 4, e4m3=e4m3)
    x, residual = inputs(T, 512)
    out, kept, idx = block.forward(x, residual)
    ex.moe.check_status(block.status)

    def wide(w, scales):
        return w.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, -1)

    w13, w2 = (wide(*block.codes13), wide(*block.codes2)) if e4m3 else (block.w13.double(), block.w2.double())
    want, want_kept = reference(block, x, residual, idx, w13, w2)
    assert off(kept, want_kept) < 2.0 ** -8
    # two roundings to E4M3 (rows, activations), the gate-up product doubles the first; else seven to bf16
    assert off(out, want) < (3 * 2.0 ** -4 / 3 ** 0.5 if e4m3 else 14 * 2.0 ** -8)


@pytest.mark.parametrize("e4m3", [False, True])
def test_step_in_a_graph(ex, e4m3):
    block = ex.Block(256, 128, 8, 2, e4m3=e4m3)
    x, residual = inputs(100, 256)
    block.forward(x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block.forward(x, residual)
    for seed in (1, 2, 3):
        a, b = inputs(100, 256, seed)
        x.copy_(a), residual.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = block.forward(x, residual)
        assert all(torch.equal(u, v) for u, v in zip(outs, want))
    ex.moe.check_status(block.status)


def test_gradients(ex):
    T, H = 300, 256
    block = ex.Block(H, 128, 8, 2)
    x, residual = inputs(T, H)
    target = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    loss, grads = block.loss_and_gradients(x, residual, target)
    ex.moe.check_status(block.status)
    _, _, idx = block.forward(x, residual)
    params = [p.double().requires_grad_() for p in block.parameters()]
    x64 = x.double().requires_grad_()
    out, kept = reference(block, x64, residual, idx, params[2], params[3], params)
    want_loss = (out + kept - target.double()).square().mean()
    want = torch.autograd.grad(want_loss, [x64, *params])
    assert abs(float(loss) - float(want_loss.detach())) < 2.0 ** -8 * float(want_loss.detach())
    for name, a, b in zip(("x", "norm", "router", "w13", "w2"), grads, want):
        assert off(a, b) < 28 * 2.0 ** -8, name


def test_gradients_while_a_captured_step_of_the_same_weights_lives(ex):
    """Training beside a serving graph of the same block, on the same stream: neither disturbs the other."""
    block = ex.Block(256, 128, 8, 2)
    x, residual = inputs(64, 256)
    block.forward(x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.forward(x, residual)[0]
    target = torch.zeros(64, 256, device="cuda")
    first = block.loss_and_gradients(x, residual, target)
    graph.replay()
    again = block.loss_and_gradients(x, residual, target)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[1], again[1]))
    assert torch.equal(out, block.forward(x, residual)[0])


@pytest.mark.parametrize("args", [[], ["--e4m3"]])
def test_program(args):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "expert_block.py"), "--tokens", "64", "--hidden", "256",
                        "--intermediate", "128", "--experts", "8", "--topk", "2", *args], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "us a step" in r.stdout and "loss" in r.stdout, r.stdout + r.stderr
