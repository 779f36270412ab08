"""Routing and rows past what 32 bits number, and biases at the ends (see test_routing.py for the tolerances)."""
import math

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_routing import check_route, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("how", [dict(), dict(groups=4, top_groups=2, group_best=2)], ids=str)
def test_biases_of_infinity(how, score):
    """+inf makes an expert chosen by every token (the lowest first), -inf by none; weights are the scores' all the same."""
    logits, b = randn(70, 32, seed=1), 0.1 * randn(32, seed=2)
    b[5] = b[20] = math.inf
    b[6] = -math.inf
    r = g.sgemm_route(logits, 4, score=score, bias=b, **how)
    check_route(r, logits, 4, score=score, bias=b, **how)
    assert (r.experts[:, 0] == 5).all() and (r.experts != 6).all()


@pytest.mark.parametrize("scale", [1e-30, 1e30, 1e-3])
@pytest.mark.parametrize("bias", [False, True])
def test_logits_of_any_size(scale, bias):
    logits = randn(60, 64, seed=3) * scale
    b = 0.1 * randn(64, seed=4) if bias else None
    check_route(g.sgemm_route(logits, 5, bias=b, renormalize=True), logits, 5, bias=b, renormalize=True)


def test_millions_of_tokens():
    T, E = (1 << 22) + 77, 8
    logits = randn(T, E, seed=5)
    r = g.sgemm_route(logits, 1)
    expert = logits.argmax(-1).int()
    assert torch.equal(r.experts[:, 0], expert)
    order = torch.argsort(expert, stable=True)
    slots = torch.empty_like(expert)
    slots[order] = torch.arange(T, dtype=torch.int32, device="cuda")
    assert torch.equal(r.slots[:, 0], slots)
    assert r.offsets[1:].tolist() == torch.cumsum(torch.bincount(expert, minlength=E), 0).tolist()
    assert g.check_status() == 0


def test_more_threads_than_one_launch_numbers():
    """Rows of an odd width, an element a thread: 2^31 and more in all, in several launches."""
    T, H = (1 << 21) + 5, 1025
    gen = torch.Generator(device="cuda").manual_seed(6)
    X = torch.randint(-128, 128, (T, H), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    slots = (T - 1 - torch.arange(T, dtype=torch.int32, device="cuda"))[:, None].contiguous()
    offsets = torch.tensor([0, T - 3], dtype=torch.int32, device="cuda")
    Y = torch.full((T + 2, H), 3.0, dtype=torch.bfloat16, device="cuda")
    g.sgemm_spread(X, slots, torch.tensor([0, T], dtype=torch.int32, device="cuda"), Y)
    assert torch.equal(Y[:T], X.flip(0)) and (Y[T:] == 0).all()
    assert torch.equal(g.sgemm_combine(Y, slots), X)
    # (the zeroed rows are the first launch's alone)
    Y.fill_(3.0)
    slots[:3] = -1
    g.sgemm_spread(X, slots, offsets, Y)
    assert torch.equal(Y[: T - 3], X[3:].flip(0)) and (Y[T - 3:] == 0).all()


def test_gradients_of_more_threads_than_one_launch_numbers():
    T, H = (1 << 25) + 7, 2
    d, Y, w = randn(T, H, seed=7), randn(T, H, seed=8), torch.rand((T, 1), device="cuda")
    slots = (T - 1 - torch.arange(T, dtype=torch.int32, device="cuda"))[:, None].contiguous()
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    dY, dw = g.sgemm_combine_grad(d, Y, slots, w, offsets)
    assert torch.equal(dY, (w * d).flip(0))  # (one product each, rounded once)
    exact = d.double() * Y.flip(0).double()
    assert ((dw[:, 0].double() - exact.sum(-1)).abs() <= 3 * 2.0 ** -24 * exact.abs().sum(-1)).all()
