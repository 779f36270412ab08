"""A layer of experts, trained in bf16 and served in 4 bits.

Rows of tokens are sent to their best experts (one each, unless more are asked for), sorted by expert, and multiplied by
that expert's two weight matrices: ``y = sum over the experts of w * relu(x W1_e) W2_e`` with the router's weights w.
Training runs the routing, the grouped products and the gradients of both, and can orthogonalise the update of the experts'
weights; afterwards the weights are quantised to MXFP4 once, and a batch and a single token are answered with 4-bit products.

    python examples/expert_layer.py [--steps N] [--choices K] [--orthogonal]

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


class Route(torch.autograd.Function):
    """Logits (T, E) to the k best experts of each token: ``(weights, offsets, slots)``, softmax scores as they are."""

    @staticmethod
    def forward(ctx, logits, k):
        r = g.sgemm_route(logits, k)
        ctx.save_for_backward(logits, r.experts)
        ctx.mark_non_differentiable(r.offsets, r.slots)
        return r.weights, r.offsets, r.slots

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, _offsets, _slots):
        logits, experts = ctx.saved_tensors
        return g.sgemm_route_grad(logits, experts, dweights.contiguous()), None


class Spread(torch.autograd.Function):
    """Tokens' rows to the places of their choices, sorted by expert."""

    @staticmethod
    def forward(ctx, X, slots, offsets):
        ctx.save_for_backward(slots)
        return g.sgemm_spread(X, slots, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        (slots,) = ctx.saved_tensors
        return g.sgemm_combine(dY.contiguous(), slots), None, None


class Combine(torch.autograd.Function):
    """The weighted sum of each token's rows."""

    @staticmethod
    def forward(ctx, Y, slots, weights, offsets):
        ctx.save_for_backward(Y, slots, weights, offsets)
        return g.sgemm_combine(Y, slots, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        Y, slots, weights, offsets = ctx.saved_tensors
        needs = (ctx.needs_input_grad[0], ctx.needs_input_grad[2])
        dY, dweights = g.sgemm_combine_grad(dout.contiguous(), Y, slots, weights, offsets, needs=needs)
        return dY, None, dweights, None


class ExpertLayer(torch.nn.Module):
    def __init__(self, experts: int, width: int, hidden: int, choices: int = 1, seed: int = 0):
        super().__init__()
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weights(*shape):
            w = torch.randn(shape, generator=gen, device="cuda") / shape[-2] ** 0.5
            return torch.nn.Parameter(w.to(torch.bfloat16))

        self.choices = choices
        self.router = torch.nn.Parameter(torch.randn((width, experts), generator=gen, device="cuda") / width ** 0.5)
        self.W1, self.W2 = weights(experts, width, hidden), weights(experts, hidden, width)

    def forward(self, x):
        weights, offsets, slots = Route.apply(x.float() @ self.router, self.choices)
        h = torch.relu(GroupedProduct.apply(Spread.apply(x, slots, offsets), self.W1, offsets))
        return Combine.apply(GroupedProduct.apply(h, self.W2, offsets), slots, weights, offsets)


class ServedLayer:
    """The same layer with its weights in 4 bits, laid out once."""

    def __init__(self, layer: ExpertLayer):
        self.router, self.choices = layer.router.detach(), layer.choices
        # (codes run along the contraction: the weights' rows are the output's columns)
        self.W1 = g.sgemm_mxfp4_quantize(layer.W1.detach().mT.contiguous())
        self.W2 = g.sgemm_mxfp4_quantize(layer.W2.detach().mT.contiguous())

    def product(self, x, W, offsets):
        return g.sgemm_mxfp4_grouped(*g.sgemm_mxfp4_quantize(x, offsets), *W, offsets)

    def __call__(self, x):
        r = g.sgemm_route(x.float() @ self.router, self.choices)
        h = torch.relu(self.product(g.sgemm_spread(x, r.slots, r.offsets), self.W1, r.offsets))
        return g.sgemm_combine(self.product(h, self.W2, r.offsets), r.slots, r.weights)


def train(layer, x, target, steps: int, rate: float = 0.05, orthogonal: bool = False):
    """Losses of plain gradient descent on the mean squared error to `target`; ``orthogonal``: the experts' weights move
    along their orthogonalised gradients."""
    losses = []
    for _ in range(steps):
        layer.zero_grad()
        loss = (layer(x).float() - target).square().mean()
        loss.backward()
        losses.append(loss.item())
        with torch.no_grad():
            for p in layer.parameters():
                if p.grad is not None:
                    d = g.sgemm_orthogonalize(p.grad) if orthogonal and p.dim() == 3 else p.grad
                    p -= (rate * d.float() * p.numel() ** 0.5 / d.float().norm().clamp(min=1e-12)
                          * p.float().abs().mean()).to(p.dtype)
    return losses


def main(steps: int = 20, tokens: int = 1000, experts: int = 8, width: int = 512, hidden: int = 1024, choices: int = 1,
         orthogonal: bool = False):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((tokens, width), generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.tanh(torch.randn((tokens, width), generator=gen, device="cuda"))
    layer = ExpertLayer(experts, width, hidden, choices)
    losses = train(layer, x, target, steps, orthogonal=orthogonal)
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
    ap.add_argument("--choices", type=int, default=1, help="experts a token")
    ap.add_argument("--orthogonal", action="store_true", help="orthogonalise the update of the experts' weights")
    a = ap.parse_args()
    main(a.steps, choices=a.choices, orthogonal=a.orthogonal)
