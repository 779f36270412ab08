"""The most matrices of a call (nothing is launched)."""
import pytest

from dense_fp32_gemm_f32_gb300 import _lib

MOST = 2 ** 27 - 1
A, B, C = 1 << 44, 1 << 46, 1 << 47  # never dereferenced


@pytest.mark.parametrize("M,N", [(1, 1), (1, 2), (2, 1), (1, 2048), (128, 2), (2, 130), (200, 3)])
def test_more_matrices_than_one_launch_numbers_are_refused(M, N):
    """(Such a call once asked for no workspace, and used one.)"""
    lib = _lib.load()
    for E in (MOST + 1, 2 ** 28, 2 ** 30):
        assert lib.sgemm_orthogonalize_workspace(_lib.TYPE_BF16, E, M, N, 5) == -1
        for workspace, size in ((None, 0), (C, 2 ** 46)):
            assert lib.sgemm_orthogonalize(_lib.TYPE_BF16, E, M, N, A, N, M * N, 5, 3.4445, -4.7750, 2.0315, 1e-7, B, N, M * N, workspace, size,
                                           None) == _lib.ERR_INVALID_ARG


def test_as_many_as_one_launch_numbers_are_not():
    assert _lib.load().sgemm_orthogonalize_workspace(_lib.TYPE_BF16, MOST, 1, 1, 5) == 0
    assert _lib.load().sgemm_orthogonalize_workspace(_lib.TYPE_BF16, MOST, 129, 129, 5) > 0
