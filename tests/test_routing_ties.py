"""Equal scores: logits of few values, biases of one value or two (see test_routing.py for the tolerances)."""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import typed
from test_routing import TYPES, check_route, randn

pytestmark = pytest.mark.gpu

GROUPS = [dict(), dict(groups=4, top_groups=2), dict(groups=8, top_groups=3, group_best=2)]


@typed(TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("how", GROUPS, ids=str)
@pytest.mark.parametrize("biases", [[0.0], [0.25], [0.0, 0.125], [-1.0, 0.0, 1.0]], ids=str)
@pytest.mark.parametrize("E", [32, 64, 256, 1024])
def test_equal_scores(E, biases, how, score, dtype):
    logits = (randn(24, E, seed=E) * 4).round() / 4
    logits[3:5] = 0
    logits[5] = -2.5
    logits[6, 1:] = -float("inf")
    logits[7] = -float("inf")
    logits[8, ::3] = -float("inf")
    logits = logits.to(dtype)
    gen = torch.Generator().manual_seed(E)
    b = torch.tensor(biases)[torch.randint(len(biases), (E,), generator=gen)].cuda()
    r = g.sgemm_route(logits, 8, score=score, bias=b, **how)
    check_route(r, logits, 8, score=score, bias=b, **how)
    if len(biases) == 1 and how.get("group_best", 1) == 1:  # (a bias of one value moves no choice)
        assert torch.equal(r.experts, g.sgemm_route(logits, 8, score=score, **how).experts)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_that_64_bits_hold_equal(score):
    """Sigmoids and softmax's small scores that round alike still follow their logits, with a bias as without one."""
    logits = torch.arange(64, device="cuda", dtype=torch.float32).flip(0).repeat(5, 1) * 8 - (0 if score == "sigmoid" else 2000)
    logits = logits[:, torch.randperm(64, generator=torch.Generator().manual_seed(1)).cuda()].contiguous()
    want = torch.sort(logits, dim=-1, descending=True).indices[:, :20].int()
    for bias in (None, torch.zeros(64, device="cuda"), torch.full((64,), 0.5, device="cuda")):
        assert torch.equal(g.sgemm_route(logits, 20, score=score, bias=bias).experts, want)
    # two biases: by logit among each one's
    bias = torch.where(torch.arange(64, device="cuda") < 32, 4.0, 0.0)
    want = want.new_tensor(torch.sort(logits[0, :32], descending=True).indices[:20].tolist())
    assert (g.sgemm_route(logits, 20, score=score, bias=bias).experts == want).all()
