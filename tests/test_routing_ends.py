"""Routing at the ends of its types' ranges (see test_routing.py for the tolerances)."""
import math

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import typed
from test_routing import HOW, TYPES, check_route, randn, scores64

INF, NAN = math.inf, math.nan


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("how", HOW, ids=str)
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("E", [20, 64, 200, 1000])
def test_gradients_that_are_not_finite_leave_experts_out_of_service_alone(E, bad, how, dtype):
    """Experts whose logit is -inf get zeros, whatever the weights' gradients; other tokens are as they would be."""
    logits = randn(9, E, seed=E, dtype=dtype)
    logits[:, ::7] = -INF
    r = g.sgemm_route(logits, 4, **how)
    d = randn(9, 4, seed=1)
    want = g.sgemm_route_grad(logits, r.experts, d, **how)
    d[3, 1] = bad
    dl = g.sgemm_route_grad(logits, r.experts, d, **how)
    assert (dl[:, ::7] == 0).all()
    keep = torch.arange(9, device="cuda") != 3
    assert torch.equal(dl[keep], want[keep])
    assert not dl[3, r.experts[3, 1].long()].isfinite()
    assert g.check_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("T,E", [(4, 32), (200, 32), (4, 256), (200, 256)])
def test_sums_of_groups_past_the_largest_float32(T, E, best, score):
    """Two biases whose sum float32 does not hold: groups are still ordered by it."""
    size = E // 4
    b = 0.1 * randn(E, seed=2)
    b[size], b[size + 1] = 3e38, 1e38
    b[2 * size + 1], b[2 * size + 3] = 3e38, 2e38
    b[3 * size], b[3 * size + 1] = -3e38, -2e38
    logits = randn(T, E, seed=3)
    how = dict(score=score, bias=b, groups=4, top_groups=1, group_best=best)
    r = g.sgemm_route(logits, 3, **how)
    check_route(r, logits, 3, **how)
    assert (r.experts[:, 0] == (size if best == 1 else 2 * size + 1)).all()
    # Now either's sum is 3e38 + 2e38 or more, and in the second's two values that 64 bits hold equal: of one bias, they follow their logits.
    b[size + 1], b[2 * size + 3] = 2e38, 3e38
    r = g.sgemm_route(logits, 3, **how)
    group = 1 if best == 1 else 2
    c, l = (scores64(logits, score) + b.double()).cpu(), logits.cpu()
    for t in range(T):
        of = sorted(range(group * size, (group + 1) * size), key=lambda e: (-c[t, e].item(), -l[t, e].item(), e))
        assert r.experts[t].tolist() == of[:3]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(3000, 64, 8), (100, 64, 8), (400, 200, 8), (120, 200, 8), (400, 40, 12)])
def test_weights_of_experts_far_below_the_largest_logit(T, E, k):
    """Chosen by their biases: scores from e^-60 to e^-87, and from there on numbers that float32 hardly holds or does not."""
    logits = randn(T, E, seed=5)
    logits[:, 0] += 13
    logits[:, 1: 1 + k] -= 2 * randn(T, k, seed=6).abs() + torch.linspace(50, 74, T, device="cuda")[:, None]
    logits[-5:, 1: 1 + k] -= 30
    logits[-2:, 1: 1 + k] *= 1e36
    b = torch.zeros(E, device="cuda")
    b[1: 1 + k] = 10.0
    r = g.sgemm_route(logits, k, bias=b)
    assert ((r.experts >= 1) & (r.experts <= k)).all()
    w = torch.gather(scores64(logits, "softmax"), 1, r.experts.long())
    assert ((r.weights.double() - w).abs() <= 2.0 ** -18 * w.amax(-1, keepdim=True) + 2.0 ** -149).all()
    assert g.check_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(4, 32), (300, 32), (4, 256), (300, 256), (4, 60)])
@pytest.mark.parametrize("how", [dict(), dict(groups=4, top_groups=1), dict(groups=4, top_groups=2, bias=1)], ids=str)
def test_logits_of_the_smallest_numbers(T, E, how):
    """Multiples of 2^-149 in float32: in order, also from group to group.  (Scores are equal; a bias of one value moves no choice.)"""
    gen = torch.Generator(device="cuda").manual_seed(E)
    units = torch.stack([torch.randperm(E, generator=gen, device="cuda") for _ in range(T)]) - E // 4
    logits = (units.double() * 2.0 ** -149).float()
    how = dict(how, bias=torch.full((E,), 0.5, device="cuda")) if "bias" in how else how
    r = g.sgemm_route(logits, 3, **how)
    by = units.clone()
    if "groups" in how:
        best = units.view(T, 4, -1).amax(-1)
        kept = torch.zeros((T, 4), dtype=torch.bool, device="cuda").scatter(1, torch.sort(best, dim=-1, descending=True).indices[:, :how["top_groups"]], True)
        by[~kept.repeat_interleave(E // 4, 1)] = -10 ** 6
    assert torch.equal(r.experts, torch.sort(by, dim=-1, descending=True).indices[:, :3].int())
    assert g.check_status() == 0
