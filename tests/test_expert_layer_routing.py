"""The example's routing: its functions together against automatic differentiation of plain operations in 64 bits, and runs with
several experts a token and orthogonalised updates."""
import math
import os
import sys

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 3])
@pytest.mark.parametrize("needs", [(True, True, True), (False, True, True), (True, False, False)])
def test_gradients_of_a_layer(k, needs):
    """Routing, spreading, grouped products and combining in float32.  Each gradient is a chain of at most four sums of
    relative error 1e-6 (see test_expert_layer.py), so 1e-4 of its norm leaves room for all."""
    from expert_layer import Combine, GroupedProduct, Route, Spread

    gen = torch.Generator(device="cuda").manual_seed(0)
    T, E, H, N = 90, 6, 40, 56
    x, w = torch.randn((T, H), generator=gen, device="cuda"), torch.randn((E, H, N), generator=gen, device="cuda")
    router = torch.randn((H, E), generator=gen, device="cuda") / 4
    R = torch.randn((T, N), generator=gen, device="cuda")
    x.requires_grad_(needs[0]), w.requires_grad_(needs[1])
    logits = (x.detach() @ router)
    logits[7:9] = -math.inf  # (padding)
    logits.requires_grad_(needs[2])
    weights, offsets, slots = Route.apply(logits, k)
    y = Combine.apply(GroupedProduct.apply(Spread.apply(x, slots, offsets), w, offsets), slots, weights, offsets)
    (y * R).sum().backward()
    experts = g.sgemm_route(logits.detach(), k).experts
    x64, w64, l64 = (t.detach().double().requires_grad_() for t in (x, w, logits))
    p = torch.nan_to_num(torch.softmax(l64, -1))
    there = experts >= 0
    at = experts.clamp(min=0).long()
    rows = torch.einsum("th,tkhn->tkn", x64, w64[at])
    (((torch.gather(p, 1, at) * there)[..., None] * rows).sum(1) * R.double()).sum().backward()
    for name, need, got, want in zip(("rows", "weights", "logits"), needs, (x.grad, w.grad, logits.grad), (x64.grad, w64.grad, l64.grad)):
        assert (got is not None) == need, name
        if need:
            want = torch.nan_to_num(want)  # (a row of -inf has no gradient)
            assert (got.double() - want).norm() <= 1e-4 * want.norm(), name


@pytest.mark.gpu
@pytest.mark.parametrize("choices,orthogonal", [(2, False), (3, True)])
def test_example_with_several_experts_a_token(choices, orthogonal):
    """Runs; 4-bit answers differ from the bf16 ones by quantisation only (see test_expert_layer.py)."""
    import expert_layer

    losses, off, off_one = expert_layer.main(steps=3, tokens=200, experts=5, width=256, hidden=384, choices=choices, orthogonal=orthogonal)
    assert all(math.isfinite(v) for v in losses)
    assert 0 < off < 0.4 and off_one < 0.6


def test_gradient_of_a_gradient_is_refused(monkeypatch):
    """(The operators are plain ones here, on the CPU.)"""
    from expert_layer import Spread

    monkeypatch.setattr(g, "sgemm_spread", lambda X, slots, offsets: X * 2)
    monkeypatch.setattr(g, "sgemm_combine", lambda Y, slots: Y * 2)
    X = torch.randn(6, 4, requires_grad=True)
    (dX,) = torch.autograd.grad(Spread.apply(X, torch.zeros(1), torch.zeros(1)).square().sum(), X, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dX.sum().backward()
