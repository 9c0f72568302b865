"""Bounded waits of the experts' and the adapter projection's kernels: one CTA keeps its first results to itself, the
others' waits for them run out after 20 ms, the call ends with MOE_ERR_TIMEOUT, and the next one, in the same workspace,
is right."""
from __future__ import annotations

import time

import pytest
import torch

pytestmark = pytest.mark.gpu
LIMIT_NS = 20_000_000


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


def rand(*shape, seed=0, std=1.0):
    return (torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) * std).bfloat16()


def experts(moe, T, H, I, E, k, e4m3):
    x, idx = rand(T, H), torch.rand(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).topk(k).indices
    weights = torch.full((T, k), 1.0 / k, device="cuda")
    w13, w2, scales = rand(E, 2 * I, H, seed=2, std=H ** -0.5), rand(E, H, I, seed=3, std=I ** -0.5), {}
    if e4m3:
        w13, w2 = ((w * 64).to(torch.float8_e4m3fn).view(torch.uint8) for w in (w13.float(), w2.float()))
        scales = dict(w13_scales=torch.full((E, 2 * I, H // 128), 1 / 64, device="cuda"),
                      w2_scales=torch.full((E, H, I // 128), 1 / 64, device="cuda"))
    ws = torch.empty(moe.moe_experts_workspace_size(T, H, I, k, E), dtype=torch.uint8, device="cuda")
    return lambda status: moe.moe_experts(x, idx, weights, w13, w2, workspace=ws, status=status, **scales)


def adapters(moe, T, K, N, L, r):
    args = (rand(T, K), rand(N, K, seed=1, std=K ** -0.5),
            torch.arange(T, device="cuda", dtype=torch.int32) * L // T, rand(L, r, K, seed=2, std=K ** -0.5),
            rand(L, N, r, seed=3, std=r ** -0.5), torch.ones(L, device="cuda"))
    ws = torch.empty(moe.moe_adapter_linear_workspace_size(T, K, N, L, r), dtype=torch.uint8, device="cuda")
    return lambda status: moe.moe_adapter_linear(*args, workspace=ws, status=status)


# few entries (every CTA plans) and many (a plan kernel); tiles that CTAs share and whole ones; two waves;
# projections sorted by adapter, whole tiles and shared ones
CASES = {
    "bf16 few": lambda moe: experts(moe, 16, 512, 256, 8, 2, False),
    "bf16 many": lambda moe: experts(moe, 300, 1024, 512, 4, 2, False),
    "bf16 two waves": lambda moe: experts(moe, 16, 7168, 512, 32, 8, False),
    "e4m3 few": lambda moe: experts(moe, 16, 512, 256, 8, 2, True),
    "e4m3 many": lambda moe: experts(moe, 200, 1024, 512, 4, 2, True),
    "e4m3 two waves": lambda moe: experts(moe, 16, 7168, 1024, 32, 8, True),
    "adapters": lambda moe: adapters(moe, 4100, 264, 4104, 5, 64),
    "adapters, shared tiles": lambda moe: adapters(moe, 600, 8328, 1064, 2, 128),
}


@pytest.mark.parametrize("cta", [0, 1])
@pytest.mark.parametrize("name", CASES)
def test_withheld_results_end_in_a_timeout(moe, name, cta):
    call = CASES[name](moe)
    status = moe.new_status()
    want = call(status)
    moe.check_status(status)
    torch.cuda.synchronize()
    with moe.test_wait_limits(LIMIT_NS, cta):
        start = time.monotonic()
        call(status)
        torch.cuda.synchronize()
        took = time.monotonic() - start
    assert int(status.item()) == moe.MOE_ERR_TIMEOUT
    assert took < 0.5        # some waits one after another, of 20 ms each
    status.zero_()
    assert torch.equal(call(status), want)
    moe.check_status(status)


def test_a_limit_alone_changes_nothing(moe):
    call, status = CASES["bf16 few"](moe), moe.new_status()
    want = call(status)
    with moe.test_wait_limits(LIMIT_NS):
        assert torch.equal(call(status), want)
    moe.check_status(status)


def test_refuses_a_cta_below_none(moe):
    with pytest.raises(moe.MoeError), moe.test_wait_limits(0, -2):
        pass
