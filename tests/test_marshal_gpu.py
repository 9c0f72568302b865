"""Checks of types, shapes and layouts in the Python functions of the gate, the experts and the adapter projection."""
from __future__ import annotations

import pytest
import torch

from combine_moe_get_gb300 import binding as moe

pytestmark = pytest.mark.gpu
BF, F32, I64, I32, U8 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.uint8


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def gate(**kw):
    d = dict(logits=zeros(4, 8)) | kw
    return moe.moe_topk_gate(d.pop("logits"), 2, **d)


def backward(**kw):
    d = dict(logits=zeros(4, 8), topk_idx=zeros(4, 2, dtype=I64), grad_weights=zeros(4, 2)) | kw
    return moe.moe_topk_gate_backward(d.pop("logits"), d.pop("topk_idx"), d.pop("grad_weights"), **d)


def experts(**kw):
    d = dict(x=zeros(4, 16, dtype=BF), topk_idx=zeros(4, 2, dtype=I64), topk_weights=zeros(4, 2),
             w13=zeros(3, 16, 16, dtype=BF), w2=zeros(3, 16, 8, dtype=BF)) | kw
    return moe.moe_experts(*[d.pop(n) for n in ("x", "topk_idx", "topk_weights", "w13", "w2")], **d)


def layer(**kw):
    d = dict(x=zeros(4, 16, dtype=BF), logits=zeros(4, 3), w13=zeros(3, 16, 16, dtype=BF), w2=zeros(3, 16, 8, dtype=BF)) | kw
    return moe.moe_layer(d.pop("x"), d.pop("logits"), 2, d.pop("w13"), d.pop("w2"), **d)


def adapter(**kw):
    d = dict(x=zeros(4, 16, dtype=BF), w=zeros(24, 16, dtype=BF), adapter_idx=zeros(4, dtype=I32),
             a=zeros(2, 8, 16, dtype=BF), b=zeros(2, 24, 8, dtype=BF), scales=zeros(2)) | kw
    return moe.moe_adapter_linear(*[d.pop(n) for n in ("x", "w", "adapter_idx", "a", "b", "scales")], **d)


@pytest.mark.parametrize("call", [gate, backward, experts, layer, adapter])
def test_accepts(call):
    call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("call, given", [
    (gate, dict(logits=(4, 8, torch.float16))),
    (gate, dict(bias=(7,))), (gate, dict(topk_idx=(4, 2))), (gate, dict(topk_weights=(2, 4))),
    (backward, dict(topk_idx=(4, 2))), (backward, dict(grad_weights=(4, 3))), (backward, dict(out=(8, 4))),
    (experts, dict(x=(4, 16))), (experts, dict(w13=(3, 15, 16, BF))), (experts, dict(w2=(3, 17, 8, BF))),
    (experts, dict(w13_scales=(3, 16, 1))), (experts, dict(topk_idx=(3, 2, I64))), (experts, dict(topk_weights=(4, 1))),
    (experts, dict(out=(4, 16))), (layer, dict(logits=(4, 4))), (layer, dict(logits=(5, 3))), (layer, dict(bias=(4,))),
    (adapter, dict(w=(24, 8, BF))), (adapter, dict(adapter_idx=(4, I64))), (adapter, dict(a=(2, 8, 24, BF))),
    (adapter, dict(b=(2, 24, 16, BF))), (adapter, dict(b=(1, 24, 8, BF))), (adapter, dict(scales=(3,))),
    (adapter, dict(out=(4, 24)))])
def test_refuses_types_and_shapes(call, given):
    made = {}
    for name, v in given.items():
        if isinstance(v, tuple):
            dtype = v[-1] if isinstance(v[-1], torch.dtype) else F32
            v = zeros(*(n for n in v if isinstance(n, int)), dtype=dtype)
        made[name] = v
    with pytest.raises(ValueError):
        call(**made)


def test_e4m3_weights_need_scales():
    codes = dict(x=zeros(4, 128, dtype=BF), w13=zeros(3, 256, 128, dtype=U8), w2=zeros(3, 128, 128, dtype=U8))
    with pytest.raises(ValueError, match="need w13_scales"):
        experts(**codes)
    experts(**codes, w13_scales=zeros(3, 256, 1), w2_scales=zeros(3, 128, 1))
    with pytest.raises(ValueError, match="w2_scales is torch.float32"):
        experts(**codes, w13_scales=zeros(3, 256, 1), w2_scales=zeros(3, 128, 2))


def test_refuses_strides():
    with pytest.raises(ValueError, match="contiguous"):
        gate(logits=zeros(8, 4).t())


def test_errors_of_the_library():
    with pytest.raises(moe.MoeError) as e:
        gate(logits=zeros(4, 1))          # two experts of one
    assert e.value.code == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoeError) as e:
        experts(workspace=zeros(16, dtype=U8))
    assert e.value.code == moe.MOE_ERR_WORKSPACE


def test_given_outputs_come_back():
    idx, w = zeros(4, 2, dtype=I64), zeros(4, 2)
    got = gate(topk_idx=idx, topk_weights=w)
    assert got[0] is idx and got[1] is w
    out = zeros(4, 24, dtype=BF)
    assert adapter(out=out) is out
    torch.cuda.synchronize()
