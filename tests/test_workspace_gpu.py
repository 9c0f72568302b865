"""One workspace, sized for the largest batch, through batches where the adapter projection changes its way."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,fewer,K,N,L,r", [(889, (888, 600, 376, 128, 1), 7168, 7168, 48, 16),
                                                (2233, (2232, 1024, 377, 100), 4096, 4096, 8, 64)])
def test_one_workspace_for_all_batches(most, fewer, K, N, L, r):
    from combine_moe_get_gb300 import binding as moe
    g = torch.Generator("cuda").manual_seed(1)
    x, w, a, b = (torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((most, K), (N, K), (L, r, K), (L, N, r)))
    idx = torch.randint(-1, L, (most,), device="cuda", generator=g, dtype=torch.int32)
    scales, status = torch.ones(L, device="cuda"), moe.new_status()
    ws = torch.empty(moe.moe_adapter_linear_workspace_size(most, K, N, L, r), dtype=torch.uint8, device="cuda")
    for T in (most, *fewer):
        args = (x[:T], w, idx[:T], a, b, scales)
        assert torch.equal(moe.moe_adapter_linear(*args, workspace=ws, status=status), moe.moe_adapter_linear(*args))
    moe.check_status(status)
