"""Calls on another stream than the current one: what a function allocates in Python, it allocates under that stream."""
from __future__ import annotations

import contextlib
from types import SimpleNamespace

import pytest
import torch

from combine_moe_get_gb300 import binding as moe

BF, I64, I32, U8 = torch.bfloat16, torch.int64, torch.int32, torch.uint8


def zeros(*shape, dtype=torch.float32, make=torch.zeros):   # not a replaced one
    return make(*shape, dtype=dtype)


def idx(T=4):
    return zeros(T, 2, dtype=I64)


X, ROWS = zeros(4, 16, dtype=BF), zeros(4, 2, dtype=I32)
W = dict(w13=zeros(3, 16, 16, dtype=BF), w2=zeros(3, 16, 8, dtype=BF))
CALLS = {
    "layout": (1, lambda **kw: moe.moe_get_layout(idx(), 8, 2, **kw)),
    "expand": (1, lambda **kw: moe.moe_get_expand_layout(idx(), zeros(9, dtype=I32), 8, **kw)),
    "dispatch": (1, lambda **kw: moe.moe_dispatch(X, idx(), None, 8, 2, ROWS, 8, **kw)),
    "quantised dispatch": (1, lambda **kw: moe.moe_dispatch(zeros(4, 128, dtype=BF), idx(), None, 8, 2, ROWS, 8,
                                                            quantize_fp8=True, **kw)),
    "layout and dispatch": (1, lambda **kw: moe.moe_layout_dispatch(X, idx(), None, 8, 2, 8, **kw)),
    "combine": (1, lambda **kw: moe.moe_combine(X, ROWS, **kw)),
    "E4M3 combine": (1, lambda **kw: moe.moe_combine_fp8(zeros(4, 128, dtype=U8), zeros(4, 1), ROWS, **kw)),
    "weighted combine": (2, lambda **kw: moe.moe_combine_ex(X, ROWS, recv_topk_weights=zeros(4, 2), **kw)),
    "gate": (1, lambda **kw: moe.moe_topk_gate(zeros(4, 8), 2, **kw)),
    "gate's gradient": (1, lambda **kw: moe.moe_topk_gate_backward(zeros(4, 8), idx(), zeros(4, 2), **kw)),
    "experts": (2, lambda **kw: moe.moe_experts(X, idx(), zeros(4, 2), **W, **kw)),
    "layer": (2, lambda **kw: moe.moe_layer(X, zeros(4, 3), 2, **W, **kw)),
    "adapters": (2, lambda **kw: moe.moe_adapter_linear(X, zeros(24, 16, dtype=BF), zeros(4, dtype=I32),
                                                        zeros(2, 8, 16, dtype=BF), zeros(2, 24, 8, dtype=BF), zeros(2), **kw)),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocates_under_the_given_stream(monkeypatch, name):
    under, made = [None], []

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        yield
        under.pop()

    def recording(make):
        def made_here(*args, **kw):
            made.append(under[-1])
            return make(*args, **kw)
        return made_here

    least, call = CALLS[name]
    side = SimpleNamespace(cuda_stream=0x1000)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for f in ("empty", "zeros"):
        monkeypatch.setattr(torch, f, recording(getattr(torch, f)))
    with pytest.raises(ValueError, match="CUDA tensors only"):   # after the allocations
        call(stream=side)
    assert len(made) >= least and set(map(id, made)) == {id(side)}, made
