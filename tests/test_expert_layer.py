"""The example: its gradients against automatic differentiation of plain products, its training, its 4-bit answers."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
def test_gradients_match_plain_products():
    """The autograd function's gradients in float32 against torch's own in 64 bits.  Each is a chain of two products of
    relative error 1e-6 at most (5e-5 of sum |a||b| bounds them; random signs make |exact| about sum / sqrt(k)), so 1e-4
    of the gradient's norm leaves room for both."""
    from expert_layer import GroupedProduct

    gen = torch.Generator(device="cuda").manual_seed(0)
    T, E, K, N, o = 120, 3, 72, 96, [0, 50, 50, 120]
    X = torch.randn((T, K), generator=gen, device="cuda", requires_grad=True)
    W = torch.randn((E, K, N), generator=gen, device="cuda", requires_grad=True)
    R = torch.randn((T, N), generator=gen, device="cuda")
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    (torch.relu(GroupedProduct.apply(X, W, offsets)) * R).sum().backward()
    x, w = X.detach().double().requires_grad_(), W.detach().double().requires_grad_()
    y = torch.cat([x[o[e]: o[e + 1]] @ w[e] for e in range(E)])
    (torch.relu(y) * R.double()).sum().backward()
    for got, want in ((X.grad, x.grad), (W.grad, w.grad)):
        assert (got.double() - want).norm() <= 1e-4 * want.norm()


@pytest.mark.gpu
def test_example_trains_and_serves():
    """Training lowers the loss; 4-bit answers differ from the bf16 ones by quantisation only: about 0.1 relative a
    product's operand (a 4-bit value is at most 1/4 off, 0.1 in the mean square), two products of two operands each."""
    import expert_layer

    losses, off, off_one = expert_layer.main(steps=8, tokens=300, experts=5, width=256, hidden=384)
    assert losses[-1] < losses[0]
    assert 0 < off < 0.4 and off_one < 0.6
