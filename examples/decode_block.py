"""A mixture-of-experts block of a few tokens, served and tuned.

Serving (`Block.step`): the requests' rows go through a projection that all of
them share, each with its own low-rank adapter beside it (moe_adapter_linear);
the router's product gives the logits; gate and experts follow in one call
(moe_layer). The block owns the workspace and the status word; nothing in a step
waits for the GPU, so a CUDA graph may hold it.

Tuning (`tune_router`): the gate as an autograd function (moe_topk_gate and
moe_topk_gate_backward), here with a cost per expert for its loss.

    python examples/decode_block.py [--tokens 16] [--hidden 1024] [--e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_moe_get_gb300 import binding as moe  # noqa: E402


class TopkGate(torch.autograd.Function):
    """logits -> (topk_idx, topk_weights), with the weights' gradient."""

    @staticmethod
    def forward(ctx, logits, num_topk, options, status):
        idx, weights = moe.moe_topk_gate(logits, num_topk, status=status, **options)
        ctx.save_for_backward(logits, idx)
        ctx.options, ctx.status = {k: v for k, v in options.items() if k != "bias"}, status
        ctx.mark_non_differentiable(idx)
        return idx, weights

    @staticmethod
    @once_differentiable   # the gradient kernel has no gradient of its own
    def backward(ctx, _, grad_weights):
        logits, idx = ctx.saved_tensors
        grad = moe.moe_topk_gate_backward(logits, idx, grad_weights.contiguous(), status=ctx.status, **ctx.options)
        return grad, None, None, None


def e4m3_rows(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """E4M3 codes (uint8) of a weight tensor [..., K] and fp32 scales [..., K/128]."""
    blocks = w.float().unflatten(-1, (-1, 128))
    scales = (blocks.abs().amax(-1) / 448.0).clamp_min(1e-12)
    codes = (blocks / scales[..., None]).to(torch.float8_e4m3fn).flatten(-2)
    return codes.view(torch.uint8), scales.contiguous()


class Block:
    """Weights and buffers of one block for steps of at most `max_tokens` rows."""

    def __init__(self, hidden, intermediate, num_experts, num_topk, num_adapters, rank, max_tokens, *, e4m3=False,
                 seed=0, device="cuda"):
        gen = torch.Generator(device).manual_seed(seed)

        def weights(*shape):
            return (torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5).bfloat16()

        self.num_topk, self.options = num_topk, dict(score="sigmoid", normalize=True, scale=2.5)
        self.w = weights(hidden, hidden)
        self.a, self.b = weights(num_adapters, rank, hidden), weights(num_adapters, hidden, rank)
        self.adapter_scales = torch.full((num_adapters,), 0.5, device=device)
        self.router = weights(num_experts, hidden)
        self.bias = torch.zeros(num_experts, device=device)
        self.w13, self.w2 = weights(num_experts, 2 * intermediate, hidden), weights(num_experts, hidden, intermediate)
        self.w13_scales = self.w2_scales = None
        if e4m3:
            self.w13, self.w13_scales = e4m3_rows(self.w13)
            self.w2, self.w2_scales = e4m3_rows(self.w2)
        # enough for smaller steps too
        need = max(moe.moe_adapter_linear_workspace_size(max_tokens, hidden, hidden, num_adapters, rank),
                   moe.moe_experts_workspace_size(max_tokens, hidden, intermediate, num_topk, num_experts))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)
        self.status = moe.new_status(torch.device(device))

    def step(self, x, adapter_idx):
        """x [T, hidden] bf16, adapter_idx int32 [T] (-1: none) -> (out, topk_idx, topk_weights)."""
        # one stream orders the two calls, so they may share the workspace
        h = moe.moe_adapter_linear(x, self.w, adapter_idx, self.a, self.b, self.adapter_scales,
                                   workspace=self.workspace, status=self.status)
        return moe.moe_layer(h, h @ self.router.T, self.num_topk, self.w13, self.w2, w13_scales=self.w13_scales,
                             w2_scales=self.w2_scales, bias=self.bias, workspace=self.workspace, status=self.status,
                             **self.options)

    def tune_router(self, x, cost, steps=8, rate=1.0):
        """Lowers the mean of cost[expert] over the choices' weights by gradient
        steps on the router; returns the loss of each step."""
        router = self.router.float().requires_grad_()
        losses = []
        for _ in range(steps):
            idx, weights = TopkGate.apply(x.float() @ router.T, self.num_topk, dict(self.options, bias=self.bias),
                                          self.status)
            loss = (weights * cost[idx]).sum(1).mean()   # every row has num_topk unmasked experts
            (grad,) = torch.autograd.grad(loss, router)
            with torch.no_grad():
                router -= rate * grad
            losses.append(float(loss.detach()))
        self.router = router.detach().bfloat16()
        return losses


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--intermediate", type=int, default=512)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--topk", type=int, default=4)
    p.add_argument("--adapters", type=int, default=8)
    p.add_argument("--rank", type=int, default=16)
    p.add_argument("--e4m3", action="store_true", help="experts' weights in E4M3")
    a = p.parse_args()
    block = Block(a.hidden, a.intermediate, a.experts, a.topk, a.adapters, a.rank, a.tokens, e4m3=a.e4m3)
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda").bfloat16()
    adapter_idx = (torch.arange(a.tokens, device="cuda", dtype=torch.int32) % (a.adapters + 1)) - 1
    for _ in range(3):
        block.step(x, adapter_idx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, idx, weights = block.step(x, adapter_idx)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    moe.check_status(block.status, "decode step")
    print(f"{a.tokens} tokens: {start.elapsed_time(end) / 20 * 1e3:.1f} us a step; first token's experts {idx[0].tolist()}, "
          f"weights {[round(v, 3) for v in weights[0].tolist()]}, |out| {float(out.float().norm()):.3f}")
    cost = torch.linspace(0.0, 1.0, a.experts, device="cuda")
    losses = block.tune_router(x, cost)
    moe.check_status(block.status, "router tuning")
    print(f"mean cost of the choices over {len(losses)} router steps: {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
