"""A mixture-of-experts block for prompts and for training: everything around a dispatch.

Serving (`Block.forward`): norm with the residual's addition (moe_add_rms_norm), router, gate, layout, an expanded
dispatch, the experts' first product (moe_grouped_linear), their activation with the router's weights (moe_swiglu), the
second product, combine. With E4M3 weights the norm makes the dispatch's codes and the activation the second product's, so
that rows travel and are multiplied in 8 bits. Numbers of rows stay on the GPU: a CUDA graph may hold a step.

Training (`Block.loss_and_gradients`): the same steps as autograd functions in bf16. A dispatch's gradient is a combine and
a combine's a dispatch; the products', the activation's, the gate's and the norm's are the library's.

    python examples/expert_block.py [--tokens 512] [--hidden 1024] [--e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_moe_get_gb300 import binding as moe  # noqa: E402
from examples.decode_block import TopkGate, e4m3_rows  # noqa: E402


class AddRmsNorm(torch.autograd.Function):
    """(x, residual, weight) -> (normed, x + residual)."""

    @staticmethod
    def forward(ctx, x, residual, weight, status):
        r = moe.moe_add_rms_norm(x, weight, residual=residual, status=status)
        ctx.save_for_backward(r.residual, weight)
        ctx.status = status
        return r.out, r.residual

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, grad_residual):
        h, weight = ctx.saved_tensors
        gx, gw = moe.moe_add_rms_norm_backward(h, weight, grad.contiguous(), grad_residual=grad_residual.contiguous(),
                                               status=ctx.status)
        return gx, gx, gw.to(weight.dtype), None


class Routing:
    """Where the rows of one batch go: the expanded layout of a choice."""

    def __init__(self, topk_idx, num_experts, status):
        self.idx, self.num_experts, self.status = topk_idx, num_experts, status
        T, k = topk_idx.shape
        self.capacity = T * k
        self.prefix = moe.moe_get_layout(topk_idx, num_experts, 1, status=status).expert_prefix
        self.rows = moe.moe_get_expand_layout(topk_idx, self.prefix, num_experts, status=status)

    def dispatch(self, x, scales=None):
        return moe.moe_dispatch(x, self.idx, None, self.num_experts, 1, self.rows, self.capacity, expand=True,
                                x_scales=scales, with_metadata=False, status=self.status)

    def combine(self, rows):
        return moe.moe_combine(rows, self.rows, status=self.status)

    def weights(self, topk_weights):
        """The router's weight of each row (every entry of the choice is valid here)."""
        return torch.zeros(self.capacity, device=topk_weights.device).index_copy(0, self.rows.flatten().long(),
                                                                                 topk_weights.flatten())


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, routing):
        ctx.routing = routing
        return routing.dispatch(x).recv_x

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        return ctx.routing.combine(grad.contiguous()), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, routing):
        ctx.routing = routing
        return routing.combine(rows)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        return ctx.routing.dispatch(grad.contiguous()).recv_x, None


class GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, prefix, status):
        ctx.save_for_backward(x, w, prefix)
        ctx.status = status
        return moe.moe_grouped_linear(x, w, prefix, status=status)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w, prefix = ctx.saved_tensors
        grad = grad.contiguous()
        gx = moe.moe_grouped_linear_grad_x(grad, w, prefix, status=ctx.status)
        gw = moe.moe_grouped_linear_grad_w(grad, x, prefix, dtype=torch.bfloat16, status=ctx.status)
        return gx, gw, None, None


class Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate_up, row_weights, status):
        ctx.save_for_backward(gate_up, row_weights)
        ctx.status = status
        return moe.moe_swiglu(gate_up, row_weights=row_weights, status=status)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        gate_up, row_weights = ctx.saved_tensors
        return (*moe.moe_swiglu_backward(gate_up, grad.contiguous(), row_weights=row_weights, status=ctx.status), None)


class Block:
    def __init__(self, hidden, intermediate, num_experts, num_topk, *, e4m3=False, seed=0, device="cuda"):
        gen = torch.Generator(device).manual_seed(seed)

        def weights(*shape):
            return (torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5).bfloat16()

        self.num_experts, self.num_topk, self.options = num_experts, num_topk, dict(score="softmax", normalize=True)
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=gen, device=device)).bfloat16()
        self.router = weights(num_experts, hidden)
        self.w13, self.w2 = weights(num_experts, 2 * intermediate, hidden), weights(num_experts, hidden, intermediate)
        self.e4m3 = e4m3
        if e4m3:
            self.codes13, self.codes2 = e4m3_rows(self.w13), e4m3_rows(self.w2)
        self.status = moe.new_status(torch.device(device))

    def forward(self, x, residual):
        """x, residual [T, hidden] bf16 -> (out, x + residual, topk_idx)."""
        s = self.status
        n = moe.moe_add_rms_norm(x, self.norm, residual=residual, quantize_fp8=self.e4m3, status=s)
        idx, topk_weights = moe.moe_topk_gate(n.out @ self.router.T, self.num_topk, status=s, **self.options)
        to = Routing(idx, self.num_experts, s)
        rows = to.prefix[-1:]
        if self.e4m3:
            (w13, s13), (w2, s2) = self.codes13, self.codes2
            d = to.dispatch(n.codes, n.scales)
            gate_up = moe.moe_grouped_linear(d.recv_x, w13, to.prefix, x_scales=d.recv_x_scales, w_scales=s13, status=s)
            h, hs = moe.moe_swiglu(gate_up, row_weights=to.weights(topk_weights), num_rows=rows, quantize_fp8=True, status=s)
            y = moe.moe_grouped_linear(h, w2, to.prefix, x_scales=hs, w_scales=s2, status=s)
        else:
            d = to.dispatch(n.out)
            gate_up = moe.moe_grouped_linear(d.recv_x, self.w13, to.prefix, status=s)
            h, _ = moe.moe_swiglu(gate_up, row_weights=to.weights(topk_weights), num_rows=rows, status=s)
            y = moe.moe_grouped_linear(h, self.w2, to.prefix, status=s)
        return to.combine(y), n.residual, idx

    def parameters(self):
        return [self.norm, self.router, self.w13, self.w2]

    def loss_and_gradients(self, x, residual, target):
        """Mean square error of out + residual to `target`, and the gradients of x and of parameters()."""
        s = self.status
        x, (norm, router, w13, w2) = x.detach().requires_grad_(), [p.detach().requires_grad_() for p in self.parameters()]
        n, kept = AddRmsNorm.apply(x, residual, norm, s)
        idx, topk_weights = TopkGate.apply(n @ router.T, self.num_topk, self.options, s)
        to = Routing(idx, self.num_experts, s)
        rows = Dispatch.apply(n, to)
        h = Swiglu.apply(GroupedLinear.apply(rows, w13, to.prefix, s), to.weights(topk_weights), s)
        out = Combine.apply(GroupedLinear.apply(h, w2, to.prefix, s), to)
        loss = (out.float() + kept.float() - target).square().mean()
        return loss.detach(), torch.autograd.grad(loss, [x, norm, router, w13, w2])


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--intermediate", type=int, default=512)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--topk", type=int, default=4)
    p.add_argument("--e4m3", action="store_true", help="experts' weights and their rows in E4M3")
    a = p.parse_args()
    block = Block(a.hidden, a.intermediate, a.experts, a.topk, e4m3=a.e4m3)
    gen = torch.Generator("cuda").manual_seed(1)
    x, residual = (torch.randn(a.tokens, a.hidden, generator=gen, device="cuda").bfloat16() for _ in range(2))
    for _ in range(3):
        block.forward(x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, idx = block.forward(x, residual)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    moe.check_status(block.status, "step")
    print(f"{a.tokens} tokens: {start.elapsed_time(end) / 20 * 1e3:.1f} us a step; first token's experts {idx[0].tolist()}, "
          f"|out| {float(out.float().norm()):.3f}")
    loss, grads = block.loss_and_gradients(x, residual, torch.zeros(a.tokens, a.hidden, device="cuda"))
    moe.check_status(block.status, "training step")
    print(f"loss {float(loss):.4f}; gradients' norms {[round(float(g.float().norm()), 5) for g in grads]}")


if __name__ == "__main__":
    main()
