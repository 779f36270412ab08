"""Choices whose values lie near one another, and every form of the choice, against 64 bits (see test_routing.py for the
tolerances).

``exact`` is the definition for many tokens at once: values in 64 bits, logits where one bias for all makes these the order.  It
is taken twice, with two ways to write the scores, whose roundings differ; a token where the two choose otherwise is one that 64
bits do not decide, and is left out (there are next to none).
"""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import typed
from test_routing import TYPES, randn, scores64
from test_routing_many import some_logits

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def scores_otherwise(l, score):
    l = l.double()
    if score == "sigmoid":
        return torch.exp(torch.nn.functional.logsigmoid(l))
    return torch.exp(l - torch.logsumexp(torch.where((l == -INF).all(-1, keepdim=True), 0.0, l), -1, keepdim=True))


def choose(s, l, k, bias, groups, top_groups, group_best):
    c = s if bias is None else s + bias.double()
    closed = (l == -INF) | (c == -INF)
    # (every order below: NaN first, then the largest, the lowest index of equal ones)
    order = lambda v: torch.sort(torch.where(v.isnan(), NAN, v), dim=-1, descending=True, stable=True).indices  # noqa: E731
    one_bias = bias is None or bool((bias == bias[0]).all() and bias[0].isfinite())
    sums = groups > 1 and group_best == 2
    by = torch.where(closed, -INF, l.double() if one_bias and not sums else c)
    if groups > 1:
        T, E = c.shape
        best = torch.sort(by.view(T, groups, -1), dim=-1, descending=True).values[..., :group_best]
        value = torch.where(best[..., 0] == -INF, -INF, torch.where(best == -INF, 0.0, best).sum(-1))
        kept = torch.zeros((T, groups), dtype=torch.bool, device=c.device).scatter(1, order(value)[:, :top_groups], True)
        closed = closed | ~kept.repeat_interleave(E // groups, 1)
    if one_bias and sums:  # (values that 64 bits hold equal still have an order, unless they are NaN)
        by = torch.where(c.isnan(), c, l.double())
    by = torch.where(closed, -INF, by)
    first = order(by)[:, :k]
    return torch.where(torch.gather(closed, 1, first), -1, first).int()


def exact(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_best=1, **_):
    """(experts, which tokens 64 bits decide)."""
    top_groups = groups if top_groups is None else top_groups
    some = [choose(s(logits, score), logits, k, bias, groups, top_groups, group_best) for s in (scores64, scores_otherwise)]
    return some[0], (some[0] == some[1]).all(-1)


def check_choice(logits, k, least=0.99, **how):
    r = g.sgemm_route(logits, k, **how)
    experts, decided = exact(logits, k, **how)
    assert decided.double().mean() >= least
    wrong = (r.experts != experts).any(-1) & decided
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[:3].flatten().tolist())
    assert g.check_status() == 0
    return r, experts, decided


def near_ties(T, E, score, open_=None, seed=0):
    """Tokens of one logit row, and a bias that brings its values to 1/2 but for the bias's rounding (2^-26)."""
    l = randn(1, E, seed=seed)
    if open_ is not None:
        closed = torch.ones(E, dtype=torch.bool, device="cuda")
        closed[torch.randperm(E, generator=torch.Generator().manual_seed(seed))[:open_].cuda()] = False
        l[:, closed] = -INF
    b = (0.5 - scores64(l, score))[0].float()
    return l.expand(T, E).contiguous(), b


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [3, 700])  # (a warp or four lanes a token, where the number of experts leaves the choice)
@pytest.mark.parametrize("E,k,open_", [(2, 1, None), (2, 2, None), (3, 1, None), (3, 2, None), (4, 2, None), (8, 3, None), (64, 1, 2), (64, 2, 3),
                                       (128, 1, 2), (256, 1, 2), (256, 2, 3), (1024, 1, 3), (36, 9, 10)])
def test_ties_of_a_few_experts(E, k, open_, T, score):
    """A few values that differ in their last bits alone: a grid from the least to the largest has them far apart.  60 rows of
    logits, each with its own bias."""
    seen = 0
    for seed in range(60):
        logits, b = near_ties(T, E, score, open_, seed)
        r = g.sgemm_route(logits, k, score=score, bias=b)
        experts, decided = exact(logits[:1], k, score=score, bias=b)
        if decided.all():
            seen += 1
            assert (r.experts == experts).all(), (seed, r.experts[0].tolist(), experts.tolist())
    assert seen >= 50 and g.check_status() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("E,groups,top,k", [(4, 2, 1, 1), (6, 3, 2, 2), (16, 2, 1, 3), (32, 4, 2, 4), (64, 8, 3, 6), (128, 4, 2, 8), (256, 8, 4, 8),
                                            (256, 2, 1, 8), (60, 3, 1, 2)])
def test_ties_of_groups(E, groups, top, k, T, best, score):
    seen = 0
    for seed in range(25):
        logits, b = near_ties(T, E, score, None, seed)
        if seed % 2:  # (one or two in service in each group)
            keep = torch.arange(E, device="cuda") % (E // groups) < 1 + seed % 4 // 2
            logits[:, ~keep] = -INF
            b = (0.5 - scores64(logits[:1], score))[0].float()
        how = dict(score=score, bias=b, groups=groups, top_groups=top, group_best=best)
        r = g.sgemm_route(logits, k, **how)
        experts, decided = exact(logits[:1], k, **how)
        if decided.all():
            seen += 1
            assert (r.experts == experts).all(), (seed, r.experts[0].tolist(), experts.tolist())
    assert seen >= 20 and g.check_status() == 0


@typed(TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
@pytest.mark.parametrize("E,groups", [(32, 4), (64, 8), (128, 4), (256, 8), (96, 3)])
def test_a_router_that_is_nearly_uniform(E, groups, bias, score, dtype):
    """Logits of 1 + 1e-3 x and 1 + 1e-6 x: sums of two are near one another, in some groups in the second order alone."""
    logits = randn(400, E, seed=E) * torch.where(torch.arange(400, device="cuda") % 2 == 0, 1e-3, 1e-6)[:, None] + 1
    b = None if bias is None else torch.full((E,), bias, device="cuda")
    check_choice(logits.to(dtype), 4, 0.9, score=score, bias=b, groups=groups, top_groups=2, group_best=2)


HOW = [dict(), dict(score="sigmoid", bias=1, renormalize=True), dict(bias=1, renormalize=True, scale=2.5), dict(score="sigmoid", bias=0),
       dict(groups=2, top_groups=1, group_best=2), dict(groups=2, top_groups=1, bias=1, score="sigmoid"), dict(groups=4, top_groups=2, bias=1),
       dict(groups=8, top_groups=4, group_best=2, bias=1, score="sigmoid"), dict(groups=8, top_groups=3), dict(groups=4, top_groups=3, group_best=2, bias=0)]


@typed(TYPES)
@pytest.mark.parametrize("how", HOW, ids=str)
@pytest.mark.parametrize("T,E,k", [(640, 64, 8), (640, 100, 5), (640, 128, 8), (640, 192, 7), (640, 256, 8), (100, 256, 8), (640, 320, 8), (300, 64, 9)])
def test_every_form(T, E, k, how, dtype):
    """Four lanes a token with 16, 32 and 64 experts a lane, and a warp a token; groups within a lane and over two of them; ties,
    near logits, tokens and experts out of service, NaN and infinities."""
    how = dict(how)
    if E % how.get("groups", 1):
        how.update(groups=2, top_groups=1)
    if "bias" in how:
        how["bias"] = 0.1 * randn(E, seed=3) if how["bias"] else torch.full((E,), 0.25, device="cuda")
    logits = some_logits(T, E, dtype)
    r, experts, decided = check_choice(logits, k, 0.97, **how)
    # the weights, of tokens without NaN and infinity
    fine = decided & ~(logits.isnan() | (logits == INF)).any(-1)
    there = experts >= 0
    at = experts.clamp(min=0).long()
    l = logits.double()
    if how.get("renormalize"):
        x = torch.gather(l if how.get("score") != "sigmoid" else torch.nn.functional.logsigmoid(l), 1, at)
        x = torch.where(there, x, torch.where(there.any(-1, keepdim=True), -INF, 0.0))
        w = torch.softmax(x, -1) * there
    else:
        w = torch.gather(scores64(logits, how.get("score", "softmax")), 1, at) * there
    w = w * how.get("scale", 1.0)
    off = (r.weights.double() - w).abs() - 2.0 ** -18 * w.amax(-1, keepdim=True) - 2.0 ** -149
    assert (off[fine] <= 0).all()
