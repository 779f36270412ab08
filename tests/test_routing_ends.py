"""Routing at the ends of its types' ranges (see test_routing.py for the tolerances)."""
import math

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import typed
from test_routing import HOW, TYPES, check_route, randn

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
