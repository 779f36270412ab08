"""Seeded random sizes, boundaries, strides and types through every grouped and MXFP4 product, against products in 64 bits."""
import math
import random

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import TYPES, bounds_of, check, dev, forward64, operands, padded, wgrad64
from test_mxfp4 import random_mxfp4

pytestmark = pytest.mark.gpu


def _size(r, lo, hi):
    v = int(math.exp(r.uniform(math.log(lo), math.log(hi))))
    step = r.choice((1, 1, 8, 64))
    return max(lo, v - v % step if v >= step else v)


def _case(r):
    while True:
        T, E, K, N = _size(r, 1, 4000), r.choice((1, 2, 3, 7, 16, 33, 64)), _size(r, 1, 2500), _size(r, 1, 2500)
        if T * K <= 6e6 and E * K * N <= 3e7:
            break
    offsets = sorted(r.randint(0, T) for _ in range(E + 1))
    if r.random() < 0.6:
        offsets[0], offsets[-1] = 0, T
    if r.random() < 0.15:
        offsets[r.randrange(E + 1)] = r.randint(-5, T + 5)
    return T, E, K, N, offsets, r.choice(TYPES), r.random() < 0.5, r.choice(((0, 0), (0, 0), (8, 0), (3, 0), (1, 5), (4, 4)))


@pytest.mark.parametrize("seed", range(12))
def test_grouped(seed):
    r = random.Random(seed)
    for i in range(20):
        T, E, K, N, offsets, dtype, transw, (pad, shift) = case = _case(r)
        X, W = operands(T, E, K, N, dtype, 100 * seed + i, transw)
        y = g.sgemm_grouped(padded(X, pad, shift), padded(W, pad, shift), dev(offsets), transw=transw)
        check(y, *forward64(X, W, offsets, transw), str(case))
        dY = torch.randn((T, N), device="cuda").to(dtype)
        dw = g.sgemm_grouped_wgrad(padded(X, pad, shift), padded(dY, pad, shift), dev(offsets),
                                   dtype=r.choice((None, torch.float32)))
        check(dw, *wgrad64(X, dY, offsets, E), str(case))
    assert g.check_status() == 0


@pytest.mark.parametrize("seed", range(6))
def test_mxfp4(seed):
    r = random.Random(1000 + seed)
    for i in range(15):
        T, E, K, N, offsets, dtype, _, (pad, shift) = case = _case(r)
        w, sw, vw = random_mxfp4((E, N, K), 100 * seed + i, 3)
        x, o = torch.randn((T, K), device="cuda").to(dtype), dev(offsets)
        a, sa = g.sgemm_mxfp4_quantize(padded(x, pad, shift), o)
        va = g.sgemm_mxfp4_dequantize(a, sa, o, cols=K).double()
        b = bounds_of(offsets, T)
        exact = torch.zeros((T, N), dtype=torch.float64, device="cuda")
        bound = exact.clone()
        for e in range(E):
            rows = slice(b[e], b[e + 1])
            exact[rows], bound[rows] = va[rows] @ vw[e].T, va[rows].abs() @ vw[e].abs().T
        check(g.sgemm_mxfp4_grouped(a, sa, w, sw, o, dtype=dtype), exact, bound, str(case))
        a, sa = g.sgemm_mxfp4_quantize(x)
        va = g.sgemm_mxfp4_dequantize(a, sa, cols=K).double()
        check(g.sgemm_mxfp4(a, sa, w[0], sw[0], dtype=dtype), va @ vw[0].T, va.abs() @ vw[0].abs().T, str(case))
    assert g.check_status() == 0
