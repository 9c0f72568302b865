"""What the Python functions of the gate, the experts and the adapter projection refuse before any call."""
from __future__ import annotations

import pytest
import torch

from combine_moe_get_gb300 import binding as moe

BF, F32, I64, I32, U8 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.uint8


def gate(**kw):
    d = dict(logits=torch.zeros(4, 8), num_topk=2, status=torch.zeros(1, dtype=I32)) | kw
    return moe.moe_topk_gate(d.pop("logits"), d.pop("num_topk"), **d)


def backward(**kw):
    d = dict(logits=torch.zeros(4, 8), idx=torch.zeros(4, 2, dtype=I64), grad=torch.zeros(4, 2),
             status=torch.zeros(1, dtype=I32)) | kw
    return moe.moe_topk_gate_backward(d.pop("logits"), d.pop("idx"), d.pop("grad"), **d)


@pytest.mark.parametrize("call", [gate, backward])
def test_tensors_of_the_cpu(call):
    with pytest.raises(ValueError, match="CUDA tensors only"):
        call()


@pytest.mark.parametrize("call", [gate, backward])
def test_score_without_a_name(call):
    with pytest.raises(ValueError, match="score is one of"):
        call(score="tanh")


@pytest.mark.parametrize("call", [gate, backward])
def test_logits_of_one_dimension(call):
    with pytest.raises(ValueError, match="2 dimensions, not 1"):
        call(logits=torch.zeros(8))


def test_not_a_tensor():
    with pytest.raises(TypeError, match="logits is not a tensor"):
        moe.moe_topk_gate([[1.0]], 1, status=torch.zeros(1, dtype=I32))


def test_number_of_arguments():
    with pytest.raises(TypeError, match="number of arguments"):
        moe._marshal.topk_gate(1, 2)
