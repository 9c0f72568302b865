"""Calls on another stream than the current one: outputs and scratch are memory of that stream, so that nothing that the
current stream does next can be given them while the call runs."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


def rand(*shape, dtype=torch.bfloat16, seed=0):
    return torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dtype)


def cases(moe):
    x, logits = rand(24, 512), rand(24, 8, dtype=torch.float32)
    w = dict(w13=rand(8, 512, 512) / 16, w2=rand(8, 512, 256) / 16)
    idx, weights = moe.moe_topk_gate(logits, 2)
    rows = moe.moe_get_layout(idx, 8, 2).token_dst_row
    adapters = (rand(512, 512) / 16, torch.arange(24, device="cuda", dtype=torch.int32) % 5 - 1, rand(4, 16, 512) / 16,
                rand(4, 512, 16) / 4, torch.ones(4, device="cuda"))
    return {
        "gate": (0, lambda **kw: moe.moe_topk_gate(logits, 2, **kw)),
        "gradient": (0, lambda **kw: [moe.moe_topk_gate_backward(logits, idx, weights, **kw)]),
        "experts": (moe.moe_experts_workspace_size(24, 512, 256, 2, 8),
                    lambda **kw: [moe.moe_experts(x, idx, weights, **w, **kw)]),
        "layer": (moe.moe_experts_workspace_size(24, 512, 256, 2, 8),
                  lambda **kw: moe.moe_layer(x, logits, 2, **w, **kw)),
        "adapters": (moe.moe_adapter_linear_workspace_size(24, 512, 512, 4, 16),
                     lambda **kw: [moe.moe_adapter_linear(x, *adapters, **kw)]),
        "layout": (moe.moe_get_layout_workspace_size(24, 8, 2),
                   lambda **kw: [moe.moe_get_layout(idx, 8, 2, **kw).token_dst_row]),
        "dispatch": (0, lambda **kw: [moe.moe_dispatch(x, idx, weights, 8, 2, rows, 48, **kw).recv_x[:24]]),
        "combine": (0, lambda **kw: [moe.moe_combine(x.repeat(2, 1), rows, **kw)]),
    }


@pytest.mark.parametrize("name", ["gate", "gradient", "experts", "layer", "adapters", "layout", "dispatch", "combine"])
def test_memory_of_the_given_stream(moe, name):
    scratch, call = cases(moe)[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()

    def reserved():
        by_stream = {}
        for s in torch.cuda.memory_snapshot():
            by_stream[s["stream"]] = by_stream.get(s["stream"], 0) + s["total_size"]
        return by_stream

    before = reserved()
    got = call(stream=side)
    after = reserved()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    own = side.cuda_stream
    assert after.get(own, 0) - before.get(own, 0) >= scratch + sum(t.numel() * t.element_size() for t in got)
    segments = [s for s in torch.cuda.memory_snapshot() if s["stream"] == own]
    for t in got:
        assert any(s["address"] <= t.data_ptr() < s["address"] + s["total_size"] for s in segments)
