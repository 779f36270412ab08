"""Orthogonalised updates of long matrices and past what 32 bits number (see test_ortho.py for the tolerances).

A matrix that is R copies of another side by side has the same left singular vectors and singular values sqrt(R) times as
large, so that its result is R copies of the other's over sqrt(R).
"""
import math

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from dense_fp32_gemm_f32_gb300 import _lib
from test_experts import typed
from test_ortho import LIMIT, QUINTIC, TYPES, ortho64

LONGEST = 1 << 18
A, B, C = 0x10000000, 1 << 45, 1 << 46  # never dereferenced


@pytest.mark.parametrize("M, N", [(300, LONGEST + 1), (LONGEST + 1, 300), (1, LONGEST + 1)])
def test_longer_rows_are_refused(M, N):
    lib = _lib.load()
    assert lib.sgemm_orthogonalize_workspace(1, 1, M, N, 5) == -1
    assert lib.sgemm_orthogonalize_workspace(1, 1, min(M, LONGEST), min(N, LONGEST), 5) > 0
    rc = lib.sgemm_orthogonalize(1, 1, M, N, A, N, M * N, 5, 3.4445, -4.7750, 2.0315, 1e-7, B, N, M * N, C, 1 << 44, None)
    assert rc == _lib.ERR_INVALID_ARG


def randn(shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def check_copies(y, S, R):
    want = ortho64(S) / math.sqrt(R)
    # (float32 sums of more than 65536 columns: 512 at a time, copies alike, and so rounded alike, are added up N / 512 times
    # with half a step of 2^-24 of the sum so far, on average half the whole: N 2^-34 of A.  A step moves a singular value s
    # by |b s^2 + 2 c s^4| <= 1.4 times that; five steps, each with what the later ones make of it, by less than 16 times.)
    N = S.shape[-1] * R
    limit = LIMIT[y.dtype] + (N * 2.0 ** -30 if N > 65536 else 0)
    for i in {0, R // 2, R - 1}:
        off = (y[..., i, :].double() - want).norm() / want.norm()
        assert off <= limit, off.item()
    assert g.check_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [7, 128, 300])
@pytest.mark.parametrize("tall", [False, True])
@typed(TYPES)
def test_the_longest_rows(M, tall, dtype):
    S, R = randn((M, 1024), dtype, seed=M), LONGEST // 1024
    G = S.repeat(1, R)
    y = g.sgemm_orthogonalize(G.T.contiguous()).T if tall else g.sgemm_orthogonalize(G)
    check_copies(y.reshape(M, R, 1024), S, R)


@pytest.mark.gpu
@typed([torch.bfloat16])
def test_rows_farther_apart_than_32_bits_number(dtype):
    M, N, ld = 300, 2048, 1 << 23
    S = randn((M, 1024), dtype, seed=1)
    G, out = (torch.empty((M, ld), dtype=dtype, device="cuda") for _ in range(2))
    assert M * ld > 2 ** 31
    G[:, :N] = S.repeat(1, 2)
    out[:, N:N + 64] = 3
    y = g.sgemm_orthogonalize(G[:, :N], out=out[:, :N])
    check_copies(y.reshape(M, 2, 1024), S, 2)
    assert (out[:, N:N + 64] == 3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M, N", [(128, 1024), (300, 1024)])
@typed([torch.bfloat16])
def test_matrices_past_2_31_elements(M, N, dtype):
    E = (1 << 31) // (M * N) + 2
    S = randn((2, M, N), dtype, seed=2)
    y = g.sgemm_orthogonalize(S[torch.arange(E, device="cuda") & 1])
    assert y.numel() > 2 ** 31
    for e in (0, 1, E // 2, E - 2, E - 1):
        check_copies(y[e].unsqueeze(-2), S[e & 1], 1)


@pytest.mark.gpu
@typed([torch.bfloat16])
def test_a_matrix_past_2_31_elements(dtype):
    """Blocks on a diagonal, each of them copies of S: singular values as if S's norm were that of all of them."""
    blocks, R = 16, LONGEST // 16 // 1024
    S = randn((520, 1024), dtype, seed=3)
    G = torch.zeros((blocks, 520, blocks, R, 1024), dtype=dtype, device="cuda")
    for i in range(blocks):
        G[i, :, i] = S[:, None]
    y = g.sgemm_orthogonalize(G.view(blocks * 520, LONGEST)).view(G.shape)
    assert y.numel() > 2 ** 31
    a, b, c = QUINTIC
    x = S.double() / (math.sqrt(blocks) * S.double().norm())
    for _ in range(5):
        x = a * x + (b * (x @ x.T) + c * (x @ x.T) @ (x @ x.T)) @ x
    x /= math.sqrt(R)
    for i in (0, 7, blocks - 1):
        for j in (0, R - 1):
            assert (y[i, :, i, j].double() - x).norm() <= LIMIT[dtype] * x.norm()
        assert not y[i, :, (i + 1) % blocks].any()
    assert g.check_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("E, M, N", [(1, 1100, 130), (1, 500, 1100), (1, 1100, 500), (2, 1000, 1200), (2, 1200, 1000), (3, 1025, 1023), (5, 450, 900),
                                     (5, 900, 450), (1, 1600, 1500), (2, 1281, 769)])
@typed(TYPES)
def test_between_few_tiles_and_many(E, M, N, dtype):
    """Sizes on either side of where tiles get wider, and of where symmetric products take one side alone."""
    G = randn((E, M, N), dtype, seed=M)
    y, want = g.sgemm_orthogonalize(G), ortho64(G)
    off = (y.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    assert (off <= LIMIT[dtype]).all(), off.max().item()
    assert g.check_status() == 0
