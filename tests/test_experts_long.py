"""Long contractions whose products have one sign, and sums that begin with their largest product: what an accumulator cuts
or rounds away at each step adds up instead of cancelling.

The acceptance is the one of test_experts.py, the bound that the header states: 5e-5 sum |a||b|, and the output's rounding.
Where it comes from, for a contraction of K <= 2^17:
* float32, few rows: 512 additions in a row at 2^-24, 3.1e-5, and K / 4096 more.
"""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import check, dev, forward64


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert g.check_status() == 0


pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("T", [2, 7])
def test_few_rows_of_products_just_below_a_rounding(T, transw):
    """One product of 1, then products just below half of 1's spacing: added to it one by one they would all be lost."""
    K, N = 1 << 17, 10000  # (so many columns that no cluster shares a tile)
    small = (2.0 ** -24 * 0.97) ** 0.5
    X = torch.full((T, K), small, device="cuda")
    W = torch.full((1, N, K) if transw else (1, K, N), small, device="cuda")
    X[:, 0] = 1.0
    (W[0, :, 0] if transw else W[0, 0])[:] = 1.0
    exact, bound = forward64(X, W[:, :32] if transw else W[:, :, :32], [0, T], transw)
    y = g.sgemm_grouped(X, W, dev([0, T]), transw=transw)
    assert torch.equal(y, y[:, :1].expand_as(y))
    check(y[:, :32], exact, bound)
