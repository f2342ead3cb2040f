"""Train linear layers with 8-bit products and orthogonalised updates.

Every step of a layer y = x W^T (W: out x in) runs through the library:

* the weight, in 128 x 128 blocks, and the layer's input and output gradient,
  in 1 x 128 and 128 x 1 blocks from one read each, are quantised to 8 bits;
* forward y = x W^T, input gradient dx = dy W (on the same weight bytes) and
  weight gradient dW = dy^T x are block-scaled 8-bit products;
* the update is the gradient's running mean, orthogonalised by Newton-Schulz
  products, as the Muon optimiser does.

Two such layers learn a fixed random linear map; the program prints the loss
as it falls.

    python examples/train_linear.py [--steps 60] [--tokens 2048] [--width 1024]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_matrix_multiplication_output_gb300 as tg  # noqa: E402


class Linear(torch.autograd.Function):
    """y = x W^T with both products' operands and both gradients in 8 bits."""

    @staticmethod
    def forward(ctx, x, weight):
        (xq, xs), by_token = tg.quantize_fp8_pair(x)   # along in; along tokens, for dW
        wq, ws = tg.quantize_fp8(weight, block="tile")
        ctx.saved = by_token, wq, ws
        return tg.matmul_fp8(xq, xs, wq, ws, op_b="t", out_dtype=torch.bfloat16)

    @staticmethod
    def backward(ctx, dy):
        (xq, xs), wq, ws = ctx.saved
        (gq, gs), (tq, ts) = tg.quantize_fp8_pair(dy.contiguous())
        dx = tg.matmul_fp8(gq, gs, wq, ws, op_b="n", out_dtype=torch.bfloat16)
        dw = tg.matmul_fp8(tq, ts, xq, xs, op_a="t", op_b="n", out_dtype=torch.float32)
        return dx, dw


class Muon:
    """w <- w - lr * sqrt(max(1, rows / cols)) * orthogonalised running mean of
    the gradient, for matrices."""

    def __init__(self, params, lr=0.02, momentum=0.9):
        self.params, self.lr, self.momentum = list(params), lr, momentum
        self.mean = [torch.zeros_like(p) for p in self.params]
        self.work = [torch.empty(tg.gemm_newton_schulz_workspace_size(1, *p.shape),
                                 dtype=torch.uint8, device=p.device) for p in self.params]

    @torch.no_grad()
    def step(self):
        for p, m, work in zip(self.params, self.mean, self.work):
            m.mul_(self.momentum).add_(p.grad)
            # (a direction: BF16's bits are enough, and the products for them cost a third)
            update = tg.newton_schulz(p.grad.add(m, alpha=self.momentum), out_dtype=torch.bfloat16,
                                      workspace=work)
            p.add_(update, alpha=-self.lr * max(1.0, p.shape[0] / p.shape[1]) ** 0.5)
            p.grad = None


def train(steps=60, tokens=2048, width=1024, hidden=768, lr=0.02, seed=0, report=None):
    """Losses of a run: a layer of hidden x width and one of width x hidden
    that together learn a random map (two layers, so that the input gradient
    is used)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    target = normal(width, width) / width ** 0.5
    w1 = torch.nn.Parameter(normal(hidden, width) / width ** 0.5)
    w2 = torch.nn.Parameter(normal(width, hidden) / hidden ** 0.5)
    optimiser = Muon([w1, w2], lr=lr)
    losses = []
    for step in range(steps):
        x = normal(tokens, width).to(torch.bfloat16)
        want = x.float() @ target.t()
        y = Linear.apply(Linear.apply(x, w1), w2)
        loss = (y.float() - want).square().mean()
        loss.backward()
        optimiser.step()
        losses.append(loss.detach())
        if report and (step % 10 == 0 or step == steps - 1):
            report(step, float(losses[-1]))
    rc = tg.gemm_device_status(torch.cuda.current_stream().cuda_stream)
    if rc != 0:
        raise RuntimeError(tg.error_string(rc))
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=768)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args()
    tg.load_library(build_if_missing=True)
    train(a.steps, a.tokens, a.width, a.hidden, a.lr,
          report=lambda i, v: print(f"step {i:4d}  loss {v:.4f}", flush=True))


if __name__ == "__main__":
    main()
