"""The example's gate as an autograd function."""
from __future__ import annotations

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_second_derivative_is_refused(monkeypatch):
    """It is not there: without an error it would be taken as zero."""
    import decode_block
    moe = decode_block.moe
    # stand-ins of the kernels on the CPU: weights are the first logits' softmax
    monkeypatch.setattr(moe, "moe_topk_gate", lambda l, k, **kw: (torch.arange(k).expand(len(l), k), l[:, :k].softmax(1)))
    monkeypatch.setattr(moe, "moe_topk_gate_backward", lambda l, idx, g, **kw: torch.ones_like(l) * g.sum())
    logits = torch.randn(3, 5, requires_grad=True)
    _, weights = decode_block.TopkGate.apply(logits, 2, {}, None)
    (grad,) = torch.autograd.grad((weights ** 2).sum(), logits, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (grad * logits).sum().backward()
