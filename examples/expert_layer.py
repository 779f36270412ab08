"""A layer of experts, trained in bf16 and served in 4 bits.

Rows of tokens are sent to their best expert each, sorted by expert, and multiplied by that expert's two weight
matrices: ``y = w * relu(x W1_e) W2_e`` with the router's weight w.  Training runs the grouped products and both of their
gradients; afterwards the weights are quantised to MXFP4 once, and a batch and a single token are answered with 4-bit
products.

    python examples/expert_layer.py [--steps N]

Prints the loss before and after training, and how far the 4-bit answers are from the bf16 ones.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_gemm_f32_gb300 as g  # noqa: E402


class GroupedProduct(torch.autograd.Function):
    """Rows sorted by expert times their expert's weights (E, K, N)."""

    @staticmethod
    def forward(ctx, X, W, offsets):
        ctx.save_for_backward(X, W, offsets)
        return g.sgemm_grouped(X, W, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, W, offsets = ctx.saved_tensors
        dY = dY.contiguous()
        dX = g.sgemm_grouped(dY, W, offsets, transw=True) if ctx.needs_input_grad[0] else None
        dW = g.sgemm_grouped_wgrad(X, dY, offsets) if ctx.needs_input_grad[1] else None
        return dX, dW, None


def route(x, router):
    """Each row's expert and its weight: ``(order, offsets, weight)``, order sorting the rows by expert."""
    p = torch.softmax(x.float() @ router, -1)
    weight, expert = p.max(-1)
    expert, order = torch.sort(expert, stable=True)
    offsets = torch.zeros(router.shape[1] + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = torch.cumsum(torch.bincount(expert, minlength=router.shape[1]), 0)
    return order, offsets, weight[order, None]


class ExpertLayer(torch.nn.Module):
    def __init__(self, experts: int, width: int, hidden: int, seed: int = 0):
        super().__init__()
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weights(*shape):
            w = torch.randn(shape, generator=gen, device="cuda") / shape[-2] ** 0.5
            return torch.nn.Parameter(w.to(torch.bfloat16))

        self.router = torch.nn.Parameter(torch.randn((width, experts), generator=gen, device="cuda") / width ** 0.5)
        self.W1, self.W2 = weights(experts, width, hidden), weights(experts, hidden, width)

    def forward(self, x):
        order, offsets, weight = route(x, self.router)
        h = torch.relu(GroupedProduct.apply(x[order], self.W1, offsets))
        y = GroupedProduct.apply(h, self.W2, offsets) * weight.to(x.dtype)
        return torch.zeros_like(y).index_copy(0, order, y)


class ServedLayer:
    """The same layer with its weights in 4 bits, laid out once."""

    def __init__(self, layer: ExpertLayer):
        self.router = layer.router.detach()
        # (codes run along the contraction: the weights' rows are the output's columns)
        self.W1 = g.sgemm_mxfp4_quantize(layer.W1.detach().mT.contiguous())
        self.W2 = g.sgemm_mxfp4_quantize(layer.W2.detach().mT.contiguous())

    def product(self, x, W, offsets):
        return g.sgemm_mxfp4_grouped(*g.sgemm_mxfp4_quantize(x, offsets), *W, offsets)

    def __call__(self, x):
        order, offsets, weight = route(x, self.router)
        h = torch.relu(self.product(x[order], self.W1, offsets))
        y = self.product(h, self.W2, offsets) * weight.to(x.dtype)
        return torch.zeros_like(y).index_copy(0, order, y)


def train(layer, x, target, steps: int, rate: float = 0.05):
    """Losses of plain gradient descent on the mean squared error to `target`."""
    losses = []
    for _ in range(steps):
        layer.zero_grad()
        loss = (layer(x).float() - target).square().mean()
        loss.backward()
        losses.append(loss.item())
        with torch.no_grad():
            for p in layer.parameters():
                if p.grad is not None:
                    p -= (rate * p.grad.float() * p.numel() ** 0.5 / p.grad.float().norm().clamp(min=1e-12)
                          * p.float().abs().mean()).to(p.dtype)
    return losses


def main(steps: int = 20, tokens: int = 1000, experts: int = 8, width: int = 512, hidden: int = 1024):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, width), generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.tanh(torch.randn((tokens, width), generator=gen, device="cuda"))
    layer = ExpertLayer(experts, width, hidden)
    losses = train(layer, x, target, steps)
    with torch.no_grad():
        served = ServedLayer(layer)
        y, y4, one = layer(x).float(), served(x).float(), served(x[:1]).float()
    assert g.check_status() == 0
    off = ((y4 - y).norm() / y.norm()).item()
    off_one = ((one - y[:1]).norm() / y[:1].norm()).item()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps; 4-bit answers off by {off:.3f} (batch), {off_one:.3f} (one token)")
    return losses, off, off_one


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    main(ap.parse_args().steps)
