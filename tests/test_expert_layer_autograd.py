"""The example's autograd function: no gradient is computed that nobody asked for, and none of a gradient."""
import os
import sys

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("needs", [(True, True), (False, True), (True, False)])
def test_only_the_gradients_asked_for(needs, monkeypatch):
    """(The products themselves are plain ones here, on the CPU.)"""
    from expert_layer import GroupedProduct

    calls = []

    def grouped(X, W, offsets, transw=False):
        calls.append("dX" if transw else "forward")
        return X @ (W[0].T if transw else W[0])

    def wgrad(X, dY, offsets):
        calls.append("dW")
        return (X.T @ dY)[None]

    monkeypatch.setattr(g, "sgemm_grouped", grouped)
    monkeypatch.setattr(g, "sgemm_grouped_wgrad", wgrad)
    X, W = torch.randn(6, 4, requires_grad=needs[0]), torch.randn(1, 4, 5, requires_grad=needs[1])
    GroupedProduct.apply(X, W, torch.tensor([0, 6], dtype=torch.int32)).sum().backward()
    assert calls == ["forward"] + [n for n, want in zip(("dX", "dW"), needs) if want]
    assert (X.grad is not None, W.grad is not None) == needs


def test_gradient_of_a_gradient_is_refused(monkeypatch):
    from expert_layer import GroupedProduct

    monkeypatch.setattr(g, "sgemm_grouped", lambda X, W, offsets, transw=False: X @ (W[0].T if transw else W[0]))
    monkeypatch.setattr(g, "sgemm_grouped_wgrad", lambda X, dY, offsets: (X.T @ dY)[None])
    X, W = torch.randn(6, 4, requires_grad=True), torch.randn(1, 4, 5, requires_grad=True)
    y = GroupedProduct.apply(X, W, torch.tensor([0, 6], dtype=torch.int32))
    (dX,) = torch.autograd.grad(y.square().sum(), X, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dX.sum().backward()
