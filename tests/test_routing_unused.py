"""Slots from offsets[E] on: rows there hold zeros, whichever thread comes last.  (Combinations read them all the same: they do
not know offsets.)"""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import typed
from test_routing import TYPES, randn

pytestmark = pytest.mark.gpu


@typed(TYPES)
@pytest.mark.parametrize("T,k,H", [(5, 2, 8), (3000, 1, 33), (2000, 4, 512), (700, 3, 4096), (40, 8, 136)])
@pytest.mark.parametrize("share", [0.0, 0.5, 1.0])
def test_slots_past_the_boundaries(T, k, H, share, dtype):
    R = T * k
    used = int(share * R)
    offsets = torch.tensor([0, used // 2, used], dtype=torch.int32, device="cuda")
    slots = torch.randperm(R, generator=torch.Generator().manual_seed(T)).int().cuda().view(T, k)
    X, w = randn(T, H, seed=1, dtype=dtype), torch.rand((T, k), device="cuda") + 0.5
    rows = torch.empty((R, H), dtype=dtype, device="cuda")
    weighted = torch.empty((R, H), device="cuda")
    for j in range(k):
        rows[slots[:, j].long()] = X
        weighted[slots[:, j].long()] = w[:, j, None] * X.float()
    rows[used:], weighted[used:] = 0, 0
    Y = randn(R, H, seed=2, dtype=dtype)
    dw = g.sgemm_combine_grad(X, Y, slots, w, offsets, needs=(False, True))[1]
    for _ in range(5):
        assert torch.equal(g.sgemm_spread(X, slots, offsets, torch.full_like(rows, 3.0)), rows)
        dY, again = g.sgemm_combine_grad(X, Y, slots, w, offsets)
        assert torch.equal(dY, weighted.to(dtype))  # (one product in float32, rounded)
        assert torch.equal(again, dw) and (dw != 0).all()
    assert g.check_status() == 0
