"""The grouped products where their kernels differ (pairs of CTAs, single ones, clusters that share a tile's reduction),
over long offsets, in CUDA graphs, on two streams at once, and where their waits run out."""
from __future__ import annotations

import os
import subprocess
import sys
import time

import pytest
import torch

from test_grouped_gpu import BF, DEV, close, codes, normal, prefix_of, values

pytestmark = pytest.mark.gpu
LIMIT_NS = 20_000_000


@pytest.fixture(scope="module")
def moe():
    from combine_moe_get_gb300 import binding
    return binding


# counts, K, N: many tiles for pairs; few, with a long reduction, for clusters of 8, 4 and 2; single CTAs; reductions that
# do not divide by the cluster; rows for several tiles, and one
WAYS = {
    "pairs": ([130, 0, 257, 64, 300, 31, 511, 7], 264, 4104),
    "cluster of 8": ([100], 7168, 512),
    "cluster of 4": ([32, 0, 32, 31, 33], 7168, 264),
    "cluster of 2": ([2048], 4104, 512),
    "one row": ([0, 1, 0], 7168, 1048),
    "uneven parts": ([3, 90], 2120, 392),
    "single": ([10, 3, 0, 25, 1], 1000, 2056),
    "several tiles": ([300, 129], 1288, 256),
}


def operands(name, e4m3=False):
    counts, K, N = WAYS[name]
    K = -(-K // 128) * 128 if e4m3 else K
    gen = torch.Generator(DEV).manual_seed(len(name))
    p = prefix_of(counts, 2)
    M, E = p[-1] + 3, len(counts)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    if e4m3:
        return p, prefix, codes(gen, M, K), codes(gen, E, N, K)
    return p, prefix, normal(gen, M, K), normal(gen, E, N, K, std=K ** -0.5), normal(gen, M, N)


@pytest.mark.parametrize("name", WAYS)
def test_bf16(moe, name):
    p, prefix, x, w, g = operands(name)
    K, N, status = x.shape[1], w.shape[1], moe.new_status()
    out, gx = torch.full_like(g, 7.0), torch.full_like(x, 7.0)
    moe.moe_grouped_linear(x, w, prefix, out=out, status=status)
    moe.moe_grouped_linear_grad_x(g, w, prefix, out=gx, status=status)
    assert torch.equal(moe.moe_grouped_linear(x, w, prefix, out=torch.full_like(g, 7.0)), out)
    moe.check_status(status)
    for t in (out, gx):
        assert (t[: p[0]] == 7).all() and (t[p[-1]:] == 7).all()
    for e in range(len(p) - 1):
        r = slice(p[e], p[e + 1])
        xe, ge, we = x[r].double(), g[r].double(), w[e].double()
        close(out[r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)
        close(gx[r], ge @ we, ge.abs() @ we.abs(), N, 2.0 ** -8)


@pytest.mark.parametrize("name", WAYS)
def test_gradient_of_rows_over_the_long_side(moe, name):
    """The reduction of grad_x is over N: the same sizes with K and N in each other's place."""
    counts, N, K = WAYS[name]
    gen = torch.Generator(DEV).manual_seed(len(name))
    p = prefix_of(counts)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    g, w = normal(gen, p[-1], N), normal(gen, len(counts), N, K, std=N ** -0.5)
    gx = moe.moe_grouped_linear_grad_x(g, w, prefix)
    for e in range(len(counts)):
        r = slice(p[e], p[e + 1])
        ge, we = g[r].double(), w[e].double()
        close(gx[r], ge @ we, ge.abs() @ we.abs(), N, 2.0 ** -8)


@pytest.mark.parametrize("name", WAYS)
def test_e4m3(moe, name):
    p, prefix, (x, xs), (w, ws) = operands(name, True)
    status = moe.new_status()
    out = torch.full((x.shape[0], w.shape[1]), 7.0, dtype=BF, device=DEV)
    moe.moe_grouped_linear(x, w, prefix, x_scales=xs, w_scales=ws, out=out, status=status)
    moe.check_status(status)
    assert (out[: p[0]] == 7).all() and (out[p[-1]:] == 7).all()
    for e in range(len(p) - 1):
        r = slice(p[e], p[e + 1])
        xe, we = values(x[r], xs[r]), values(w[e], ws[e])
        close(out[r], xe @ we.T, xe.abs() @ we.abs().T, x.shape[1], 2.0 ** -8)


# counts, K, N: weights' gradients whose tiles are few and rows many; an expert without rows and one with fewer blocks
# than the cluster has CTAs
WEIGHTS = {
    "pairs, 2 of them": ([6001], 1272, 1528),
    "pairs, 4 of them": ([11998, 3], 1016, 504),
    "single": ([130, 128, 0, 1, 127] * 3, 520, 392),
    "2 of them": ([3500], 2040, 512),
    "4 of them": ([5001], 1000, 504),
    "8 of them": ([5000], 512, 264),
    "uneven experts": ([9000, 0, 40, 65], 136, 72),
}


def weights_operands(name):
    counts, K, N = WEIGHTS[name]
    gen = torch.Generator(DEV).manual_seed(len(name))
    p = prefix_of(counts, 5)
    return p, torch.tensor(p, dtype=torch.int32, device=DEV), normal(gen, p[-1] + 9, K), normal(gen, p[-1] + 9, N)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("name", WEIGHTS)
def test_weights_shared(moe, name, dtype):
    p, prefix, x, g = weights_operands(name)
    E, N, K, status = len(p) - 1, g.shape[1], x.shape[1], moe.new_status()
    # rows of no expert, which the first and last block of an expert's rows go on into
    x[: p[0]], x[p[-1]:], g[: p[0]], g[p[-1]:] = float("nan"), float("inf"), float("inf"), float("nan")
    out = torch.full((E, N, K), 7.0, dtype=dtype, device=DEV)
    moe.moe_grouped_linear_grad_w(g, x, prefix, out=out, status=status)
    again = torch.randn(E, N, K, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(dtype)
    start = again.clone()
    moe.moe_grouped_linear_grad_w(g, x, prefix, out=again, accumulate=True, status=status)
    assert torch.equal(moe.moe_grouped_linear_grad_w(g, x, prefix, dtype=dtype), out)
    moe.check_status(status)
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    for e in range(E):
        r = slice(p[e], p[e + 1])
        rows = p[e + 1] - p[e]
        if rows == 0:
            assert not out[e].any() and torch.equal(again[e], start[e])
            continue
        xe, ge, s = x[r].double(), g[r].double(), start[e].double()
        want, size = ge.T @ xe, ge.abs().T @ xe.abs()
        close(out[e], want, size, rows, half)
        close(again[e], want + s, size + s.abs(), rows + 1, half)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_shared_weights_follow_the_prefix(moe, dtype):
    """One capture of a shared gradient serves rows for one expert, for all, for none, and a prefix with a bad end."""
    _, prefix, x, g = weights_operands("uneven experts")
    E, M, status = prefix.numel() - 1, x.shape[0], moe.new_status()
    out = torch.empty(E, g.shape[1], x.shape[1], dtype=dtype, device=DEV)
    call = lambda: moe.moe_grouped_linear_grad_w(g, x, prefix, out=out, accumulate=False, status=status)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    for p in ([0, M, M, M, M], [0, 1, 2, 3, 4], [M] * 5, [0, 63, 128, 2000, M], [0, 5, 5, 5, M]):
        prefix.copy_(torch.tensor(p, dtype=torch.int32))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for e in range(E):
            xe, ge = x[p[e]: p[e + 1]].double(), g[p[e]: p[e + 1]].double()
            close(out[e], ge.T @ xe, ge.abs().T @ xe.abs(), max(1, p[e + 1] - p[e]), half)
    moe.check_status(status)
    prefix[-1] = M + 1
    graph.replay()
    assert int(status.item()) == moe.MOE_ERR_BAD_PREFIX


def test_shared_weights_at_once(moe):
    calls = []
    for name in WEIGHTS:
        _, prefix, x, g = weights_operands(name)
        calls.append(lambda x=x, g=g, prefix=prefix, **kw: moe.moe_grouped_linear_grad_w(g, x, prefix, **kw))
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [c(stream=s) for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_e4m3_scales_far_apart(moe):
    """Blocks whose scales differ by 2^40, and scales at no 16-byte boundary."""
    gen = torch.Generator(DEV).manual_seed(9)
    p = [0, 40, 200]
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    (x, xs), (w, ws) = codes(gen, 200, 1024), codes(gen, 2, 72, 1024)
    xs, ws = xs * 2.0 ** torch.randint(-20, 20, xs.shape, device=DEV, generator=gen), ws * 2.0 ** -30
    odd = [torch.empty(t.numel() + 1, device=DEV)[1:].view(t.shape).copy_(t) for t in (xs, ws)]
    for a, b in ((xs, ws), odd):
        out = moe.moe_grouped_linear(x, w, prefix, x_scales=a, w_scales=b)
        for e in range(2):
            r = slice(p[e], p[e + 1])
            xe, we = values(x[r], xs[r]), values(w[e], ws[e])
            close(out[r], xe @ we.T, xe.abs() @ we.abs().T, 1024, 2.0 ** -8)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_weights_offsets_beyond_32_bits(moe, dtype):
    """Weights of 2^32 elements and more, rows at both ends."""
    E, N, K = 66, 8192, 8192
    gen = torch.Generator(DEV).manual_seed(10)
    p = [0, 5] + [5] * (E - 2) + [12]
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, g = normal(gen, 12, K), normal(gen, 12, N)
    w = torch.empty(E, N, K, dtype=BF, device=DEV)
    w[0], w[-1] = normal(gen, N, K, std=K ** -0.5), normal(gen, N, K, std=K ** -0.5)
    out, gx = moe.moe_grouped_linear(x, w, prefix), moe.moe_grouped_linear_grad_x(g, w, prefix)
    for e, r in ((0, slice(0, 5)), (E - 1, slice(5, 12))):
        xe, ge, we = x[r].double(), g[r].double(), w[e].double()
        close(out[r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)
        close(gx[r], ge @ we, ge.abs() @ we.abs(), N, 2.0 ** -8)
    del w
    gw = moe.moe_grouped_linear_grad_w(g, x, prefix, dtype=dtype)
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    for e, r in ((0, slice(0, 5)), (E - 1, slice(5, 12))):
        xe, ge = x[r].double(), g[r].double()
        close(gw[e], ge.T @ xe, ge.abs().T @ xe.abs(), 7, half)
    assert not gw[1: E - 1].any()


def test_rows_offsets_beyond_32_bits(moe):
    M, K, N = 280_000, 64, 8192   # 2.3 * 10^9 outputs
    gen = torch.Generator(DEV).manual_seed(11)
    p = [0, 3, M - 300, M]
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, w = normal(gen, M, K), normal(gen, 3, N, K, std=K ** -0.5)
    out = moe.moe_grouped_linear(x, w, prefix)
    for e in range(3):
        r = slice(max(p[e], p[e + 1] - 300), p[e + 1])
        xe, we = x[r].double(), w[e].double()
        close(out[r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)
    gx = moe.moe_grouped_linear_grad_x(out, w, prefix)
    r = slice(M - 300, M)
    close(gx[r], out[r].double() @ w[2].double(), out[r].double().abs() @ w[2].double().abs(), N, 2.0 ** -8)


def test_a_graph_follows_the_prefix(moe):
    """Numbers of rows stay on the device: a captured call serves whatever the prefix says when it runs."""
    gen = torch.Generator(DEV).manual_seed(12)
    E, M, K, N = 6, 700, 520, 264
    x, g, w = normal(gen, M, K), normal(gen, M, N), normal(gen, E, N, K, std=K ** -0.5)
    prefix = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    out, gx, gw = torch.empty(M, N, dtype=BF, device=DEV), torch.empty(M, K, dtype=BF, device=DEV), torch.empty(E, N, K, device=DEV)
    status = moe.new_status()

    def step():
        moe.moe_grouped_linear(x, w, prefix, out=out, status=status)
        moe.moe_grouped_linear_grad_x(g, w, prefix, out=gx, status=status)
        moe.moe_grouped_linear_grad_w(g, x, prefix, out=gw, status=status)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in ([700, 0, 0, 0, 0, 0], [1, 2, 3, 4, 5, 6], [0, 0, 300, 250, 0, 0], [116] * 6):
        prefix.copy_(torch.tensor(prefix_of(counts), dtype=torch.int32))
        for t in (out, gx, gw):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, gx, gw)]
        n = sum(counts)
        assert (got[0][n:] == 7).all() and (got[1][n:] == 7).all()
        for t in (out, gx, gw):
            t.fill_(7)
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, gx, gw)))
        for e in range(E):
            r = slice(sum(counts[:e]), sum(counts[: e + 1]))
            xe, ge, we = x[r].double(), g[r].double(), w[e].double()
            close(got[0][r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)
            close(got[2][e], ge.T @ xe, ge.abs().T @ xe.abs(), max(1, counts[e]), 2.0 ** -24)
    moe.check_status(status)


def test_two_calls_at_once(moe):
    calls = []
    for name in ("pairs", "cluster of 8", "single"):
        _, prefix, x, w, g = operands(name)
        calls.append((lambda x=x, w=w, prefix=prefix, **kw: moe.moe_grouped_linear(x, w, prefix, **kw)))
        calls.append((lambda g=g, w=w, prefix=prefix, **kw: moe.moe_grouped_linear_grad_x(g, w, prefix, **kw)))
    want = [c() for c in calls]
    rows = [slice(2, -3)] * len(calls)   # those of no expert are not written
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [c(stream=s) for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a[r], b[r]) for a, b, r in zip(got, want, rows))


@pytest.mark.parametrize("E,counts", [(8192, {0: 3, 31: 1, 32: 40, 5000: 17, 8191: 200}), (40, {e: 1 for e in range(40)}),
                                      (2, {0: 5000, 1: 2300})])
def test_many_experts_and_many_rows(moe, E, counts):
    K, N = 72, 264
    gen = torch.Generator(DEV).manual_seed(E)
    p = prefix_of([counts.get(e, 0) for e in range(E)])
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, g, w = normal(gen, p[-1], K), normal(gen, p[-1], N), normal(gen, E, N, K, std=K ** -0.5)
    status = moe.new_status()
    out = moe.moe_grouped_linear(x, w, prefix, status=status)
    gx = moe.moe_grouped_linear_grad_x(g, w, prefix, status=status)
    gw = moe.moe_grouped_linear_grad_w(g, x, prefix, status=status)
    moe.check_status(status)
    for e in counts:
        r = slice(p[e], p[e + 1])
        xe, ge, we = x[r].double(), g[r].double(), w[e].double()
        close(out[r], xe @ we.T, xe.abs() @ we.abs().T, K, 2.0 ** -8)
        close(gx[r], ge @ we, ge.abs() @ we.abs(), N, 2.0 ** -8)
        close(gw[e], ge.T @ xe, ge.abs().T @ xe.abs(), counts[e], 2.0 ** -24)
    empty = [e for e in range(E) if e not in counts]
    assert not gw[empty].any()


@pytest.mark.parametrize("name", ["pairs", "cluster of 8", "cluster of 4", "single"])
@pytest.mark.parametrize("last", [-1, 10 ** 9])
def test_a_bad_end_of_the_prefix_is_seen(moe, name, last):
    p, prefix, x, w, g = operands(name)
    prefix[-1] = last
    for call in (lambda s: moe.moe_grouped_linear(x, w, prefix, status=s),
                 lambda s: moe.moe_grouped_linear_grad_x(g, w, prefix, status=s),
                 lambda s: moe.moe_grouped_linear_grad_w(g, x, prefix, status=s)):
        status = moe.new_status()
        call(status)
        assert int(status.item()) == moe.MOE_ERR_BAD_PREFIX


def test_a_rank_takes_its_part_of_the_prefix(moe):
    """The received rows of all ranks in one buffer, each rank's weights by themselves."""
    gen = torch.Generator(DEV).manual_seed(16)
    counts, K, N = [5, 0, 130, 9, 64, 31], 136, 72
    p = prefix_of(counts)
    prefix = torch.tensor(p, dtype=torch.int32, device=DEV)
    x, w = normal(gen, p[-1], K), normal(gen, 6, N, K, std=K ** -0.5)
    want = moe.moe_grouped_linear(x, w, prefix)
    got = torch.zeros_like(want)
    for rank in range(3):
        moe.moe_grouped_linear(x, w[2 * rank: 2 * rank + 2], prefix[2 * rank: 2 * rank + 3], out=got)
    assert torch.equal(got, want)


FIRST_IN_CAPTURE = """
import torch
from combine_moe_get_gb300 import binding as moe
gen = torch.Generator("cuda").manual_seed(1)
x, w, g = (torch.randn(*s, device="cuda", generator=gen).bfloat16() for s in ((300, 256), (3, 2048, 256), (300, 2048)))
prefix = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
gu, n = torch.randn(300, 512, device="cuda").bfloat16(), torch.ones(256, device="cuda")
status = moe.new_status()
moe.moe_topk_gate(torch.zeros(1, 8, device="cuda"), 1, status=status)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def step():
    r = moe.moe_add_rms_norm(x, n, quantize_fp8=True, status=status)
    return (moe.moe_grouped_linear(x, w, prefix, status=status), moe.moe_grouped_linear_grad_x(g, w, prefix, status=status),
            moe.moe_grouped_linear_grad_w(g, x, prefix, status=status), moe.moe_swiglu(gu, status=status)[0],
            moe.moe_swiglu_backward(gu, x, status=status)[0], r.out, r.codes,
            *moe.moe_add_rms_norm_backward(x, n, x, status=status))
with torch.cuda.graph(graph):
    outs = step()
graph.replay()
torch.cuda.synchronize()
moe.check_status(status)
assert all(torch.equal(a, b) for a, b in zip(outs, step()))
print("captured")
"""


def test_the_first_call_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_traced(moe):
    """Every new kernel leaves records in the tracing build."""
    from combine_moe_get_gb300 import build
    lib = moe.load_library(build.build_trace())
    records, count = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    p, prefix, x, w, g = operands("uneven parts")
    gu, ones = normal(torch.Generator(DEV).manual_seed(17), 40, 512), torch.ones(256, device=DEV)
    h = gu[:, :256].contiguous()
    with moe.using(lib):
        moe.trace_enable(records, count)
        try:
            moe.moe_grouped_linear(x, w, prefix)
            moe.moe_swiglu(gu)
            moe.moe_swiglu_backward(gu, h)
            moe.moe_add_rms_norm(h, ones)
            moe.moe_add_rms_norm_backward(h, ones, h)
            torch.cuda.synchronize()
        finally:
            moe.trace_enable(None, None)
    seen = {moe.TRACE_KERNELS[k] for k in moe.trace_read(records, count)["kernel"]}
    assert seen == {"grouped", "swiglu", "swiglu_backward", "norm", "norm_backward", "norm_weight"}


# ------------------------------------------------------------------ waits

def withheld_cases(moe):
    for name in ("pairs", "cluster of 8", "single"):
        _, prefix, x, w, g = operands(name)
        yield name, lambda s, x=x, w=w, p=prefix: moe.moe_grouped_linear(x, w, p, out=torch.zeros(x.shape[0], w.shape[1], dtype=BF, device=DEV), status=s)
        yield name + ", rows", lambda s, g=g, w=w, p=prefix: moe.moe_grouped_linear_grad_x(g, w, p, out=torch.zeros(g.shape[0], w.shape[2], dtype=BF, device=DEV), status=s)
        yield name + ", weights", lambda s, g=g, x=x, p=prefix: moe.moe_grouped_linear_grad_w(g, x, p, status=s)
        _, prefix, (x, xs), (w, ws) = operands(name, True)
        yield name + ", E4M3", lambda s, x=x, xs=xs, w=w, ws=ws, p=prefix: moe.moe_grouped_linear(
            x, w, p, x_scales=xs, w_scales=ws, out=torch.zeros(x.shape[0], w.shape[1], dtype=BF, device=DEV), status=s)


@pytest.mark.parametrize("cta", [0, 1, 5])
def test_withheld_rows_of_a_shared_gradient(moe, cta):
    for name in ("pairs, 4 of them", "2 of them", "8 of them", "uneven experts"):
        _, prefix, x, g = weights_operands(name)
        status = moe.new_status()
        want = moe.moe_grouped_linear_grad_w(g, x, prefix, status=status)
        moe.check_status(status, name)
        torch.cuda.synchronize()
        with moe.test_wait_limits(LIMIT_NS, cta):
            start = time.monotonic()
            moe.moe_grouped_linear_grad_w(g, x, prefix, status=status)
            torch.cuda.synchronize()
            assert time.monotonic() - start < 1.0, name
        assert int(status.item()) == moe.MOE_ERR_TIMEOUT, name
        status.zero_()
        assert torch.equal(moe.moe_grouped_linear_grad_w(g, x, prefix, status=status), want), name
        moe.check_status(status, name)


@pytest.mark.parametrize("cta", [0, 1])
def test_withheld_operands_end_in_a_timeout(moe, cta):
    for name, call in withheld_cases(moe):
        status = moe.new_status()
        want = call(status)
        moe.check_status(status, name)
        torch.cuda.synchronize()
        with moe.test_wait_limits(LIMIT_NS, cta):
            start = time.monotonic()
            call(status)
            torch.cuda.synchronize()
            took = time.monotonic() - start
        assert int(status.item()) == moe.MOE_ERR_TIMEOUT, name
        assert took < 1.0, name   # some waits one after another, of 20 ms each
        status.zero_()
        assert torch.equal(call(status), want), name
        moe.check_status(status, name)
