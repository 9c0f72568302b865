"""A workspace that is sized for the largest batch is enough for every smaller one: sizes never fall as rows are added."""
from __future__ import annotations

import pytest

from combine_moe_get_gb300 import binding as moe

# ranges in which the adapter projection changes its way, and its tiles' width, back and forth
ADAPTERS = [(7168, 7168, 48, 16), (7168, 4096, 16, 64), (4096, 4096, 8, 64), (7168, 2048, 8, 16), (4096, 4096, 128, 16),
            (264, 4104, 5, 64), (64, 4096, 1000, 8), (8, 1 << 20, 4, 128), (1 << 20, 64, 8192, 8), (8200, 1064, 2, 128)]
EXPERTS = [(7168, 2048, 8, 256), (7168, 2048, 8, 32), (256, 256, 2, 16), (1160, 520, 3, 24), (512, 384, 2, 3), (64, 64, 1, 1)]


@pytest.mark.parametrize("K,N,L,r", ADAPTERS)
def test_adapter_workspace_never_falls(K, N, L, r):
    sizes = [moe.moe_adapter_linear_workspace_size(T, K, N, L, r) for T in range(1, 4500)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))
    far = [moe.moe_adapter_linear_workspace_size(T, K, N, L, r) for T in range(4499, 1 << 20, 4093)]
    assert sizes[-1] <= far[0] and all(a <= b for a, b in zip(far, far[1:]))


@pytest.mark.parametrize("H,I,k,E", EXPERTS)
def test_experts_workspace_never_falls(H, I, k, E):
    sizes = [moe.moe_experts_workspace_size(T, H, I, k, E) for T in range(1, 1025)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_a_few_rows_take_little():
    assert moe.moe_adapter_linear_workspace_size(1, 7168, 2048, 8, 16) < 1 << 20
    assert moe.moe_adapter_linear_workspace_size(128, 7168, 7168, 48, 16) < 8 << 20
