"""The operators where their plans change: two waves of experts, more sets than a warp each can count, wide tiles, many
entries to an expert, a rank's mostly masked rows, and the biased choice over long batches. Definitions and tolerances
are those of the operators' own test files."""
from __future__ import annotations

import math

import pytest
import torch

import test_adapter_gpu
import test_experts_gpu
from test_gate_gpu import make_logits, rtol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


def check_experts(moe, p):
    status = moe.new_status()
    got = p.call(moe, status=status)
    test_experts_gpu.check(got, *p.reference())
    moe.check_status(status)
    assert torch.equal(p.call(moe), got)


# Two waves take 28 K blocks of phase 1 or more to each of the SMs (4256 of them on 152), in tiles of at most 64
# columns: here groups x 28 tiles x (8 blocks of 64, or of 128 columns).
@pytest.mark.parametrize("unnamed,masked", [((), 0.0), ((4,), 0.0), ((0, 31), 0.3)])
@pytest.mark.parametrize("I,e4m3", [(512, False), (520, False), (1024, True)])
def test_two_waves_of_experts(moe, I, e4m3, unnamed, masked):
    p = test_experts_gpu.Problem(16, 7168, I, 32, 8, e4m3=e4m3, seed=I, masked=masked)
    for e in unnamed:              # an odd number of groups, or none at the ends
        p.idx[p.idx == e] = -1
    assert len(p.idx[p.idx >= 0].unique()) >= 24
    check_experts(moe, p)


@pytest.mark.parametrize("T,H,I,E,k", [(30, 128, 128, 600, 4), (3, 256, 128, 4096, 8), (200, 128, 128, 4096, 8),
                                       (70, 128, 128, 8192, 3)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_many_experts(moe, T, H, I, E, k, e4m3):
    check_experts(moe, test_experts_gpu.Problem(T, H, I, E, k, e4m3=e4m3, seed=E, masked=0.1))


@pytest.mark.parametrize("T,H,I,E,k,e4m3", [(512, 1024, 384, 3, 2, False), (1024, 2048, 264, 8, 4, False),
                                            (1000, 1160, 136, 2, 1, False), (600, 256, 256, 4, 2, True),
                                            (1024, 1152, 384, 8, 4, True)])
def test_hundreds_of_entries_to_an_expert(moe, T, H, I, E, k, e4m3):
    check_experts(moe, test_experts_gpu.Problem(T, H, I, E, k, e4m3=e4m3, seed=T + H))


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_whose_entries_are_mostly_other_ranks(moe, e4m3):
    check_experts(moe, test_experts_gpu.Problem(350, 512, 256, 32, 8, e4m3=e4m3, seed=8, masked=0.85))


@pytest.mark.parametrize("spread", ["rows", "runs"])
@pytest.mark.parametrize("shape", [(33, 64, 72, 2500, 8), (6000, 64, 4096, 3000, 8), (5000, 64, 4104, 8192, 8)])
def test_thousands_of_adapters(moe, shape, spread):
    p = test_adapter_gpu.Problem(*shape, spread=spread, seed=sum(shape))
    status = moe.new_status()
    got = p.call(moe, status=status)
    test_adapter_gpu.check(got, *p.reference())
    moe.check_status(status)
    assert torch.equal(p.call(moe), got)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(5000, 256, 8), (3000, 1000, 6), (2100, 2048, 8), (300, 8192, 8)])
def test_biased_choice_of_a_long_batch(moe, T, E, k, score, normalize):
    l = make_logits(T, E, torch.float32, E)
    l[7] = -math.inf
    l[8, 3:] = -math.inf
    g = torch.Generator().manual_seed(4)
    bias = (torch.randn(E, generator=g) * 0.3).cuda()
    bias[6] = math.nan              # never chosen
    status = moe.new_status()
    idx, w = moe.moe_topk_gate(l, k, bias=bias, score=score, normalize=normalize, status=status)
    moe.check_status(status)
    ld = l.double()
    s = torch.where(ld > -math.inf, torch.softmax(ld, 1) if score == "softmax" else torch.sigmoid(ld), 0.0)
    v = torch.where((ld > -math.inf) & ~bias.isnan(), s + bias.double(), -math.inf)
    on = idx >= 0
    assert torch.equal(on.sum(1), (v > -math.inf).sum(1).clamp_max(k))
    got = torch.where(on, v.gather(1, idx.clamp_min(0)), 0.0)
    want = v.sort(dim=1, descending=True).values[:, :k]
    off = rtol(l) + 2.0 ** -22      # both sums' rounding
    torch.testing.assert_close(got, torch.where(on, want, 0.0), rtol=off, atol=off)
    apart = idx.sort(dim=1).values
    assert bool(((apart[:, 1:] > apart[:, :-1]) | (apart[:, :-1] < 0)).all())
    rw = torch.where(on, s.gather(1, idx.clamp_min(0)), 0.0)
    rw = rw / rw.sum(1, keepdim=True).clamp_min(1e-300) if normalize else rw
    torch.testing.assert_close(w.double(), rw, rtol=rtol(l), atol=1e-30)
