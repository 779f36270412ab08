"""Hundreds of experts, most of them with few rows or none, one with many."""
import random

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import TYPES, check, dev, forward64, operands, typed, wgrad64
from test_mxfp4 import random_mxfp4

pytestmark = pytest.mark.gpu


def uneven(T, E, seed):
    """Sorted boundaries: a fifth of the rows to one expert, the others' by chance, many empty."""
    r = random.Random(seed)
    cuts = sorted(r.randint(0, T - T // 5) for _ in range(E - 2))  # (E - 1 groups)
    big = r.randrange(E)
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [T - T // 5])]
    sizes.insert(big, T // 5)
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    assert len(out) == E + 1 and out[-1] == T
    return out


@typed(TYPES)
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("T,E,K,N", [(1152, 64, 264, 392), (3, 384, 136, 200), (700, 257, 136, 200), (9000, 300, 64, 136)])
def test_products(T, E, K, N, transw, dtype):
    offsets = uneven(T, E, 1) if T > 5 else [0] * 100 + [1] * 200 + [2] + [3] * (E - 300)
    X, W = operands(T, E, K, N, dtype, 2, transw)
    check(g.sgemm_grouped(X, W, dev(offsets), transw=transw), *forward64(X, W, offsets, transw))
    dY = torch.randn((T, N), device="cuda").to(dtype)
    check(g.sgemm_grouped_wgrad(X, dY, dev(offsets)), *wgrad64(X, dY, offsets, E))
    assert g.check_status() == 0


@pytest.mark.parametrize("T,E", [(3, 384), (700, 257), (9000, 300)])
def test_mxfp4(T, E):
    K, N = 96, 136
    offsets = uneven(T, E, 3) if T > 5 else [0] * 100 + [1] * 200 + [2] + [3] * (E - 300)
    w, sw, vw = random_mxfp4((E, N, K), 4)
    x, o = torch.randn((T, K), device="cuda"), dev(offsets)
    a, sa = g.sgemm_mxfp4_quantize(x, o)
    va = g.sgemm_mxfp4_dequantize(a, sa, o, cols=K).double()
    exact = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    bound = exact.clone()
    for e in range(E):
        rows = slice(offsets[e], offsets[e + 1])
        exact[rows], bound[rows] = va[rows] @ vw[e].T, va[rows].abs() @ vw[e].abs().T
    check(g.sgemm_mxfp4_grouped(a, sa, w, sw, o, dtype=torch.float32), exact, bound)
    assert g.check_status() == 0
