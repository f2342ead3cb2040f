"""Train a layer of experts, and adapters beside a frozen projection, through the
products grouped by rows and the low-rank adapters.

* ExpertLayer: every token goes to the `top` experts of highest score.  Its copies
  are sorted by expert, multiplied by their expert's matrices (matmul_grouped,
  one call for all experts, whatever number of rows each has), and summed with the
  scores' weights.  Backward, the same call with the matrices as stored gives the
  input's gradient, and matmul_grouped_wgrad the experts'.
* AdapterLayer: a projection that stays as it is, with a low-rank adapter for each
  task (matmul_lora); a batch may mix tasks in any order.  Backward:
  matmul_lora_backward.

The program fits both to a fixed random map and prints the loss as it falls.

    python examples/train_experts.py [--steps 60] [--tokens 2048] [--width 512]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_matrix_multiplication_output_gb300 as tg  # noqa: E402


class GroupedLinear(torch.autograd.Function):
    """y[i] = x[i] @ w[g]^T for the rows of each group g; w: groups x out x in."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return tg.matmul_grouped(x, w, offsets, out_dtype=x.dtype)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = tg.matmul_grouped(dy, w, offsets, op_b="n", out_dtype=x.dtype)
        return dx, tg.matmul_grouped_wgrad(dy, x, offsets, out_dtype=w.dtype), None


class AdaptedLinear(torch.autograd.Function):
    """y_i = x_i @ w^T + scale[g] * x_i @ a[g]^T @ b[g]^T, g the row's adapter; w is frozen."""

    @staticmethod
    def forward(ctx, x, w, a, b, adapter, scale):
        ctx.save_for_backward(x, w, a, b, adapter, scale)
        return tg.matmul_lora(x, w, a, b, adapter, scale, out_dtype=x.dtype)

    @staticmethod
    def backward(ctx, dy):
        x, w, a, b, adapter, scale = ctx.saved_tensors
        dx, da, db = tg.matmul_lora_backward(dy.contiguous(), x, w, a, b, adapter, scale,
                                             out_dtype=x.dtype, grad_dtype=a.dtype)
        return dx, None, da, db, None, None


def route(scores, top):
    """(rows: each token's copies sorted by expert, offsets: the experts' first rows,
    weights: of each copy in that order)."""
    weight, expert = torch.softmax(scores, dim=-1).topk(top, dim=-1)
    order = expert.reshape(-1).argsort(stable=True)
    counts = torch.bincount(expert.reshape(-1), minlength=scores.shape[1])
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    return order // top, offsets, weight.reshape(-1)[order]


class ExpertLayer(torch.nn.Module):
    """Two matrices an expert with a SiLU between, and a router."""

    def __init__(self, experts, width, hidden, top, dtype, device="cuda"):
        super().__init__()

        def matrix(*shape):
            return torch.nn.Parameter((torch.randn(*shape, device=device) * shape[-1] ** -0.5).to(dtype))

        self.top = top
        self.router = torch.nn.Parameter(torch.randn(experts, width, device=device) * width ** -0.5)
        self.up, self.down = matrix(experts, hidden, width), matrix(experts, width, hidden)

    def forward(self, x):
        rows, offsets, weight = route(x.float() @ self.router.t(), self.top)
        h = GroupedLinear.apply(x[rows], self.up, offsets)
        y = GroupedLinear.apply(torch.nn.functional.silu(h), self.down, offsets)
        out = torch.zeros(x.shape, device=x.device)
        return out.index_add(0, rows, weight[:, None] * y.float()).to(x.dtype)


class AdapterLayer(torch.nn.Module):
    """A frozen projection with an adapter for each task."""

    def __init__(self, w, tasks, rank, dtype):
        super().__init__()
        n, k = w.shape
        self.register_buffer("w", w)
        self.register_buffer("scale", torch.full((tasks,), 2.0, device=w.device))
        self.a = torch.nn.Parameter((torch.randn(tasks, rank, k, device=w.device) * k ** -0.5).to(dtype))
        self.b = torch.nn.Parameter(torch.zeros(tasks, n, rank, device=w.device, dtype=dtype))

    def forward(self, x, adapter):
        return AdaptedLinear.apply(x, self.w, self.a, self.b, adapter, self.scale)


def train(steps=60, tokens=2048, width=512, experts=8, tasks=5, rank=16, lr=3e-3, log=print):
    """Returns the losses of every step."""
    torch.manual_seed(0)
    dtype = torch.bfloat16
    w = (torch.randn(width, width, device="cuda") * width ** -0.5).to(dtype)
    moe = ExpertLayer(experts, width, 2 * width, 2, dtype)
    adapted = AdapterLayer(w, tasks, rank, dtype)
    target = torch.randn(tasks, width, width, device="cuda") * width ** -0.5
    params = list(moe.parameters()) + list(adapted.parameters())
    opt = torch.optim.Adam(params, lr=lr)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, width, device="cuda").to(dtype)
        task = torch.randint(0, tasks, (tokens,), device="cuda", dtype=torch.int32)
        want = torch.einsum("tk,tnk->tn", x.float(), target[task.long()]) if tokens <= 256 else \
            sum(torch.where((task == t)[:, None], x.float() @ target[t].t(), 0.0) for t in range(tasks))
        loss = (moe(adapted(x, task)).float() - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {losses[-1]:.4f}")
    rc = tg.gemm_device_status(torch.cuda.current_stream().cuda_stream)
    if rc != 0:
        raise RuntimeError(tg.error_string(rc))
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--width", type=int, default=512)
    args = p.parse_args()
    train(args.steps, args.tokens, args.width)


if __name__ == "__main__":
    main()
