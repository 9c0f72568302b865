"""Tensors on several devices, or on another one than the current, are refused, and a status that is no int32 word.
(Tensors without memory stand for those of a second device.)"""
from __future__ import annotations

import inspect

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from combine_moe_get_gb300 import binding as moe

BF, F32, I64, I32, U8 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.uint8

GATE = dict(logits=(4, 8), bias=(8,), topk_idx=(4, 2, I64), topk_weights=(4, 2), status=(1, I32))
BACKWARD = dict(logits=(4, 8), topk_idx=(4, 2, I64), grad_weights=(4, 2), out=(4, 8), status=(1, I32))
EXPERTS = dict(x=(4, 128, BF), topk_idx=(4, 2, I64), topk_weights=(4, 2), w13=(3, 256, 128, U8), w2=(3, 128, 128, U8),
               w13_scales=(3, 256, 1), w2_scales=(3, 128, 1), out=(4, 128, BF), workspace=(16, U8), status=(1, I32))
LAYER = dict(EXPERTS, logits=(4, 3), bias=(3,))
ADAPTER = dict(x=(4, 16, BF), w=(24, 16, BF), adapter_idx=(4, I32), a=(2, 8, 16, BF), b=(2, 24, 8, BF), scales=(2,),
               out=(4, 24, BF), workspace=(16, U8), status=(1, I32))
CALLS = [(moe.moe_topk_gate, GATE), (moe.moe_topk_gate_backward, BACKWARD), (moe.moe_experts, EXPERTS),
         (moe.moe_layer, LAYER), (moe.moe_adapter_linear, ADAPTER)]


@pytest.fixture(autouse=True)
def no_context_for_tensors_without_memory(monkeypatch):
    """On a machine with one GPU there is none for cuda:1."""
    monkeypatch.setattr("torch._subclasses.fake_tensor.init_gpu_context", lambda device: None, raising=False)


def call(f, tensors, device_of):
    mode, args = FakeTensorMode(), {}
    with mode:
        for name, v in tensors.items():
            dtype = v[-1] if isinstance(v[-1], torch.dtype) else F32
            args[name] = torch.empty(*(n for n in v if isinstance(n, int)), dtype=dtype, device=device_of(name))
    if "num_topk" in inspect.signature(f).parameters:
        args["num_topk"] = 2
    return f(**args)


@pytest.mark.parametrize("f,tensors,name", [(f, t, n) for f, t in CALLS for n in t])
def test_one_tensor_on_another_device(f, tensors, name):
    with pytest.raises(ValueError, match="is on cuda:"):
        call(f, tensors, lambda n: "cuda:1" if n == name else "cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("f,tensors", CALLS)
def test_all_tensors_on_another_device_than_the_current(f, tensors):
    with pytest.raises(ValueError, match="tensors on cuda:1, the current device is cuda:0"):
        call(f, tensors, lambda n: "cuda:1")


@pytest.mark.parametrize("f,tensors", CALLS)
@pytest.mark.parametrize("status", [(1, U8), (1, I64), (1, F32), (0, I32)])
def test_status_of_another_type_or_without_an_element(f, tensors, status):
    """Kernels write four bytes to it."""
    with pytest.raises(ValueError, match="status is torch.int32"):
        call(f, dict(tensors, status=status), lambda n: "cuda:0")
