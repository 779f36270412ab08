"""Outputs that are zeros without a product (no rows, no contraction, no experts)."""
import ctypes

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import TYPES, dev, typed

pytestmark = pytest.mark.gpu


def nodes(call):
    """Operations on the GPU that a call records."""
    call()  # (set-up outside the capture)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = ctypes.c_size_t()
    assert ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


@typed(TYPES)
@pytest.mark.parametrize("K,N", [(8, 24), (1, 7), (5, 1)])
@pytest.mark.parametrize("layout", ["whole", "matrices apart", "rows apart", "both apart"])
def test_gradient_of_no_rows(layout, K, N, dtype):
    E = 5
    store = torch.full((E, K + 2, N + 3), 7.0, dtype=dtype, device="cuda")
    out = {"whole": torch.full((E, K, N), 7.0, dtype=dtype, device="cuda"),
           "matrices apart": torch.full((E, (K + 2) * N), 7.0, dtype=dtype, device="cuda")[:, : K * N].unflatten(1, (K, N)),
           "rows apart": torch.full((E, K, N + 3), 7.0, dtype=dtype, device="cuda")[..., :N],
           "both apart": store[:, :K, :N]}[layout]
    X, dY, o = torch.empty((0, K), dtype=dtype, device="cuda"), torch.empty((0, N), dtype=dtype, device="cuda"), dev([0] * (E + 1))
    whole = out._base if out._base is not None else out
    g.sgemm_grouped_wgrad(X, dY, o, out)
    assert not out.any()
    assert int((whole == 7).sum()) == whole.numel() - out.numel(), "padding was written"


def test_gradient_of_no_rows_is_one_operation():
    X, dY, o = torch.empty((0, 64), device="cuda"), torch.empty((0, 128), device="cuda"), dev([0] * 385)
    out = torch.empty((384, 64, 128), device="cuda")
    assert nodes(lambda: g.sgemm_grouped_wgrad(X, dY, o, out)) == 1
    wide = torch.empty((384, 64, 130), device="cuda")[..., :128]
    assert nodes(lambda: g.sgemm_grouped_wgrad(X, dY, o, wide)) == 1
