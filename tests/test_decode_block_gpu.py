"""examples/decode_block.py: the adapter projection, the gate and the experts used together."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def inputs(T, hidden, adapters):
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(T, hidden, generator=g, device="cuda").bfloat16()
    return x, torch.randint(-1, adapters, (T,), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 13])
def test_step_is_the_operators_one_after_another(example, T, e4m3):
    moe = example.moe
    block = example.Block(512, 256, 32, 4, 5, 8, 13, e4m3=e4m3)
    x, adapter = inputs(T, 512, 5)
    h = moe.moe_adapter_linear(x, block.w, adapter, block.a, block.b, block.adapter_scales)
    idx, weights = moe.moe_topk_gate(h @ block.router.T, 4, bias=block.bias, **block.options)
    out = moe.moe_experts(h, idx, weights, block.w13, block.w2, w13_scales=block.w13_scales, w2_scales=block.w2_scales)
    got = block.step(x, adapter)
    torch.cuda.synchronize()
    moe.check_status(block.status, "step")
    for a, b in zip(got, (out, idx, weights)):
        assert torch.equal(a, b)


def test_step_in_a_graph(example):
    block = example.Block(512, 256, 32, 4, 5, 8, 13)
    x, adapter = inputs(13, 512, 5)
    want = [t.clone() for t in block.step(x, adapter)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block.step(x, adapter)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_gate_as_an_autograd_function(example):
    """fp32 gradient of a product of the weights, against automatic differentiation
    of the definition in 64 bits: at most some tens of fp32 roundings of values up to 1."""
    g = torch.Generator("cuda").manual_seed(3)
    logits = torch.randn(9, 32, generator=g, device="cuda").requires_grad_()
    cost = torch.rand(9, 4, generator=g, device="cuda")
    status = example.moe.new_status(logits.device)
    options = dict(score="sigmoid", normalize=True, scale=2.5)
    idx, weights = example.TopkGate.apply(logits, 4, options, status)
    (grad,) = torch.autograd.grad((weights * cost).sum(), logits)
    exact = logits.detach().double().requires_grad_()
    s = exact.sigmoid().gather(1, idx)
    (want,) = torch.autograd.grad((2.5 * s / s.sum(1, keepdim=True) * cost.double()).sum(), exact)
    assert (grad.double() - want).abs().max() < 2.0 ** -18


def test_router_tuning_lowers_the_cost(example):
    block = example.Block(512, 256, 32, 4, 5, 8, 64)
    x, _ = inputs(64, 512, 5)
    losses = block.tune_router(x, torch.linspace(0.0, 1.0, 32, device="cuda"))
    example.moe.check_status(block.status, "tuning")
    assert all(b < a for a, b in zip(losses, losses[1:]))
