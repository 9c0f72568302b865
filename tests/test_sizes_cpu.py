"""Sizes and numbers beyond 32 bits, which the C entry points do not have, are refused and not cut. (Tensors without
memory stand for large ones.)"""
from __future__ import annotations

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from combine_moe_get_gb300 import binding as moe

BF, I64, I32 = torch.bfloat16, torch.int64, torch.int32
MORE = 2 ** 32


@pytest.fixture(scope="module")
def fake():
    mode = FakeTensorMode()

    def make(*shape, dtype=torch.float32):
        with mode:
            return torch.empty(*shape, dtype=dtype, device="cuda:0")
    return make


def gate(fake, T=4, E=8, k=2):
    return moe.moe_topk_gate(fake(T, E), k, status=fake(1, dtype=I32))


def backward(fake, T=4, E=8):
    return moe.moe_topk_gate_backward(fake(T, E), fake(T, 2, dtype=I64), fake(T, 2), status=fake(1, dtype=I32))


def experts(fake, T=4, H=16, I=8, E=3, k=2):
    return moe.moe_experts(fake(T, H, dtype=BF), fake(T, k, dtype=I64), fake(T, k), fake(E, 2 * I, H, dtype=BF),
                           fake(E, H, I, dtype=BF), status=fake(1, dtype=I32), workspace=fake(16))


def layer(fake, T=4, H=16, I=8, E=3, k=2):
    return moe.moe_layer(fake(T, H, dtype=BF), fake(T, E), k, fake(E, 2 * I, H, dtype=BF), fake(E, H, I, dtype=BF),
                         status=fake(1, dtype=I32), workspace=fake(16))


def adapter(fake, T=4, K=16, N=24, L=2, r=8):
    return moe.moe_adapter_linear(fake(T, K, dtype=BF), fake(N, K, dtype=BF), fake(T, dtype=I32), fake(L, r, K, dtype=BF),
                                  fake(L, N, r, dtype=BF), fake(L), status=fake(1, dtype=I32), workspace=fake(16))


SIZES = [(gate, "T"), (gate, "E"), (backward, "T"), (backward, "E"), (experts, "T"), (experts, "H"), (experts, "I"),
         (experts, "E"), (experts, "k"), (layer, "T"), (layer, "H"), (layer, "I"), (layer, "E"), (adapter, "T"),
         (adapter, "K"), (adapter, "N"), (adapter, "L"), (adapter, "r")]


@pytest.mark.parametrize("call,size", SIZES)
@pytest.mark.parametrize("n", [2 ** 31, MORE + 8])
def test_sizes_beyond_32_bits(fake, call, size, n):
    with pytest.raises(ValueError, match=f"size of {n} does not fit in 32 bits"):
        call(fake, **{size: n})


@pytest.mark.parametrize("call", [gate, layer])
@pytest.mark.parametrize("k", [MORE + 2, 2 - MORE, 2 ** 31, 2 ** 80])
def test_a_number_beyond_32_bits(fake, call, k):
    with pytest.raises(OverflowError):
        call(fake, k=k)


@pytest.mark.parametrize("i", range(5))
def test_workspace_of_sizes_beyond_32_bits(i):
    for size, good in ((moe.moe_experts_workspace_size, (4, 16, 8, 2, 3)),
                       (moe.moe_adapter_linear_workspace_size, (4, 16, 24, 2, 8))):
        assert size(*good) > 0
        assert size(*(n + MORE * (j == i) for j, n in enumerate(good))) == 0
        assert size(*(n - MORE * (j == i) for j, n in enumerate(good))) == 0
