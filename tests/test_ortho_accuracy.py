"""How exact orthogonalised updates are, beyond what test_ortho.py asks.

A bf16 result is rounded once, from values that are as exact as float32's.  Let z be what is rounded and x the exact value: the
nearest bf16 value to z is no farther from z than the nearest one to x is, so that the result is off by at most half a step of bf16 at
x and 2 |z - x|.  What it is off beyond half a step has therefore at most twice the norm of z - x.

That norm: 2^-18 of the result's for five steps of the usual polynomial (see test_ortho.py).  For more steps, and polynomials that raise
errors, it is compared with the same steps whose products are float32's, and may be 16 times theirs: a sum in an accumulator is cut to
24 bits up to 32 times, 2^-20 on average, where a product in float32 is rounded by 2^-24.
"""
import math

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from dense_fp32_gemm_f32_gb300 import _lib
from test_experts import typed
from test_ortho import A, B, C, QUINTIC, ortho64, update

TYPES = [torch.float32, torch.bfloat16, torch.float16]
DIGITS = {torch.float32: 24, torch.bfloat16: 8, torch.float16: 11}
SMALLEST = {torch.float32: -149, torch.bfloat16: -133, torch.float16: -24}


def beyond_rounding(y, exact):
    """The norm of what each result is off beyond half a step of its type, over the exact one's."""
    step = torch.ldexp(torch.ones_like(exact), (torch.frexp(exact).exponent - DIGITS[y.dtype]).clamp(min=SMALLEST[y.dtype]))
    off = ((y.double() - exact).abs() - step / 2).clamp(min=0)
    return off.flatten(-2).norm(dim=-1) / exact.flatten(-2).norm(dim=-1)


def float32_steps(G, steps, coefficients):
    a, b, c = coefficients
    X = G.double()
    X = (X / (X.square().sum((-2, -1), keepdim=True).sqrt() + 1e-7)).float()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    for _ in range(steps):
        S = X @ X.mT
        X = a * X + (b * S + c * (S @ S)) @ X
    return X.mT if tall else X


SHAPES = [(1, 20, 30), (1, 96, 128), (2, 300, 128), (1, 100, 1024), (1, 128, 2048), (1, 3000, 100), (1, 129, 129), (2, 300, 520), (1, 1000, 700),
          (2, 1025, 1023), (2, 1000, 2000), (3, 2000, 1000)]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("rank", [0, 4])
@pytest.mark.parametrize("E,M,N", SHAPES)
def test_a_result_is_rounded_once(E, M, N, rank, dtype):
    G = update(E, M, N, dtype, seed=M + N, rank=rank)
    off = beyond_rounding(g.sgemm_orthogonalize(G), ortho64(G))
    assert (off <= 2 * 2.0 ** -18).all(), off.max().item()
    assert g.check_status() == 0


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("rank", [0, 3])
@pytest.mark.parametrize("M,N", [(100, 200), (256, 384), (700, 640)])
@pytest.mark.parametrize("coefficients,steps", [((3.0, -1.0, 0.0), 6), ((3.0, -1.0, 0.0), 8), (QUINTIC, 10), (QUINTIC, 20), ((2.0, -1.5, 0.5), 30)], ids=str)
def test_many_steps_and_polynomials_that_raise_errors(coefficients, steps, M, N, rank, dtype):
    G = update(1, M, N, dtype, seed=1, rank=rank)
    exact = ortho64(G, steps, coefficients)
    usual = ((float32_steps(G, steps, coefficients).double() - exact).norm() / exact.norm()).item()
    off = beyond_rounding(g.sgemm_orthogonalize(G, steps=steps, coefficients=coefficients), exact).item()
    assert off <= 2 * (16 * usual + 2.0 ** -18), (off, usual)
    assert g.check_status() == 0


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("rank", [1, 2, 8, 30])
@pytest.mark.parametrize("M,N", [(60, 64), (100, 300), (2000, 128), (300, 400), (512, 512), (1000, 1300)])
def test_matrices_of_low_rank(M, N, rank, dtype):
    """Whole numbers that every type holds: nothing but the roundings of the steps in the other directions."""
    gen = torch.Generator(device="cuda").manual_seed(M + rank)
    u, v = (torch.randint(-2, 3, s, generator=gen, device="cuda").float() for s in ((M, rank), (rank, N)))
    G = (u @ v).to(dtype)[None]
    assert torch.equal(G[0].float(), u @ v)
    exact = ortho64(G)
    usual = ((float32_steps(G, 5, QUINTIC).double() - exact).norm() / exact.norm()).item()
    off = beyond_rounding(g.sgemm_orthogonalize(G), exact).item()
    assert off <= 2 * (16 * usual + 2.0 ** -18), (off, usual)
    assert off <= 2.0 ** -11
    assert g.check_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [0, 4])
@pytest.mark.parametrize("E,M,N", SHAPES + [(8, 1000, 3000)])
def test_quick_products(E, M, N, rank):
    """Nine roundings of operands, each 2^-12 / sqrt(3) in the mean, in parts of the polynomial of up to 8: below 2^-8 of the norm
    (see test_ortho.py)."""
    G = update(E, M, N, torch.bfloat16, seed=M + N, rank=rank)
    y = g.sgemm_orthogonalize(G, quick=True)
    assert (beyond_rounding(y, ortho64(G)) <= 2 * 2.0 ** -8).all()
    assert torch.equal(y, g.sgemm_orthogonalize(G, torch.empty_like(G), quick=True))
    assert g.check_status() == 0


def test_quick_products_are_for_bf16_alone():
    lib = _lib.load()
    for t, rc in ((_lib.TYPE_F32, _lib.ERR_INVALID_ARG), (_lib.TYPE_F16, _lib.ERR_INVALID_ARG), (3, _lib.ERR_INVALID_ARG), (_lib.TYPE_BF16, _lib.OK)):
        t += _lib.ORTHO_QUICK
        assert lib.sgemm_orthogonalize(t, 0, 16, 32, 0, 32, 512, 5, *QUINTIC, 1e-7, 0, 32, 512, 0, 0, None) == rc
        assert (lib.sgemm_orthogonalize_workspace(t, 1, 300, 500, 5) > 0) == (rc == _lib.OK)
    size = [lib.sgemm_orthogonalize_workspace(t, 3, 512, 1000, 5) for t in (_lib.TYPE_BF16, _lib.TYPE_BF16 + _lib.ORTHO_QUICK)]
    assert size[0] - size[1] == 2 * 3 * 512 * 512  # (the second plane of an operand)
    small = lib.sgemm_orthogonalize_workspace(_lib.TYPE_BF16 + _lib.ORTHO_QUICK, 2, 200, 256, 5) - 256
    assert lib.sgemm_orthogonalize(_lib.TYPE_BF16 + _lib.ORTHO_QUICK, 2, 200, 256, A, 256, 51200, 5, *QUINTIC, 1e-7, B, 256, 51200, C, small,
                                   None) == _lib.ERR_INVALID_ARG


@pytest.mark.gpu
@typed([torch.float32, torch.float16])
def test_quick_products_of_other_types_are_refused(dtype):
    G = update(1, 20, 30, dtype)
    for out in (None, torch.empty_like(G)):
        with pytest.raises(ValueError):
            g.sgemm_orthogonalize(G, out, quick=True)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("eps", [1e-7, 2.0 ** -140, 1e-60, 1e-100, 1e-300, 5e-324])
@pytest.mark.parametrize("M,N", [(20, 30), (100, 300), (300, 200)])
def test_zeros_stay_zeros_with_the_smallest_eps(M, N, eps, dtype):
    G = update(3, M, N, dtype, seed=1)
    G[1] = 0
    y = g.sgemm_orthogonalize(G, eps=eps)
    assert (y[1] == 0).all()
    assert (beyond_rounding(y[[0, 2]], ortho64(G[[0, 2]], eps=eps)) <= 2 * 2.0 ** -18).all()
    assert g.sgemm_orthogonalize(G, eps=0.0)[1].isnan().all()
    assert g.check_status() == 0


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("ratio", [0.9, 1.0, 3.0, 60.0, 1e3, 1e5, 1e8, 1e14, 1e25])
@pytest.mark.parametrize("M,N", [(60, 64), (100, 300), (300, 128), (300, 400), (700, 640)])
def test_norms_far_below_eps(M, N, ratio, dtype):
    """Small X, whose bits the result keeps: relative to its own norm, however small that is."""
    G = update(3, M, N, dtype, seed=M, size=1.0)
    G[1] *= 2.0 ** -10
    eps = ratio * G[0].double().norm().item()
    for steps, coefficients in ((5, QUINTIC), (1, QUINTIC), (12, (2.0, -1.5, 0.5)), (3, (1.0, 0.0, 0.0))):
        y, exact = g.sgemm_orthogonalize(G, eps=eps, steps=steps, coefficients=coefficients), ortho64(G, steps, coefficients, eps)
        assert (beyond_rounding(y, exact) <= 2 * 2.0 ** -18).all(), (steps, coefficients, beyond_rounding(y, exact).tolist())
        if dtype == torch.bfloat16 and steps == 5:
            assert (beyond_rounding(g.sgemm_orthogonalize(G, eps=eps, quick=True), exact) <= 2 * 2.0 ** -8).all()
    assert g.check_status() == 0
