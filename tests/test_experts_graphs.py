"""Recorded calls whose operands come from several streams: a product may begin its set-up beside the kernel before it, and has to
wait for all of what it reads."""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import check, dev, forward64

pytestmark = pytest.mark.gpu


def test_operands_quantised_on_two_streams():
    T, E, K, N = 3000, 2, 2048, 520
    x, w, o = torch.randn((T, K), device="cuda"), torch.randn((E, N, K), device="cuda"), dev([0, 1300, T])
    g.sgemm_mxfp4_grouped(*g.sgemm_mxfp4_quantize(x, o), *g.sgemm_mxfp4_quantize(w), o)  # (set-up)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        b = g.sgemm_mxfp4_quantize(w, stream=side)  # (the longer one)
        a = g.sgemm_mxfp4_quantize(x, o)
        main.wait_stream(side)
        y = g.sgemm_mxfp4_grouped(*a, *b, o, dtype=torch.float32)
    for seed in range(3):
        x.normal_()
        w.normal_()
        graph.replay()
        torch.cuda.synchronize()
        va, vb = g.sgemm_mxfp4_dequantize(*a, o).double(), g.sgemm_mxfp4_dequantize(*b).double()
        exact, bound = torch.cat([va[:1300] @ vb[0].T, va[1300:] @ vb[1].T]), torch.cat([va[:1300].abs() @ vb[0].abs().T, va[1300:].abs() @ vb[1].abs().T])
        want = g.sgemm_mxfp4_quantize(x, o)
        assert torch.equal(want[0], a[0])
        check(y, exact, bound)
    assert g.check_status() == 0


@pytest.mark.parametrize("recorded", [False, True])
def test_products_after_a_join(recorded):
    """Rows and weights written on two other streams just before the product."""
    T, E, K, N, offsets = 2000, 2, 1032, 264, [0, 900, 2000]
    X, W, o = torch.zeros((T, K), device="cuda"), torch.zeros((E, K, N), device="cuda"), dev(offsets)
    src = [(torch.randn_like(X), torch.randn_like(W)) for _ in range(2)]
    X16, W16 = X.to(torch.bfloat16), W.to(torch.bfloat16)
    g.sgemm_grouped(X16, W16, o)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    from_x, from_w = torch.empty_like(X), torch.empty_like(W)

    def step():
        main = torch.cuda.current_stream()
        for s, dst, frm in ((s1, X16, from_x), (s2, W16, from_w)):
            s.wait_stream(main)
            with torch.cuda.stream(s):
                torch.cuda._sleep(200000)
                dst.copy_(frm)
        main.wait_stream(s1)
        main.wait_stream(s2)
        return g.sgemm_grouped(X16, W16, o)

    if recorded:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = step()
    for x, w in src:
        from_x.copy_(x)
        from_w.copy_(w)
        if recorded:
            graph.replay()
        else:
            y = step()
        torch.cuda.synchronize()
        check(y, *forward64(x.to(torch.bfloat16), w.to(torch.bfloat16), offsets))
    assert g.check_status() == 0
