"""Operands that the caller drops while a call on another stream has yet to read them."""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import TYPES, dev, typed

pytestmark = pytest.mark.gpu


def on_a_busy_stream(call, *operands):
    """call(*copies of the operands, stream) on a stream that is asleep; the copies go out of scope and their memory is
    asked for again, and written, before it wakes.  (Once on an idle stream first: a kernel's first launch may wait for the
    GPU.)"""
    for cycles in (1, 100_000_000):
        s = torch.cuda.Stream()
        copies = [t.clone() for t in operands]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(cycles)
        result = call(*copies, s)
        shapes = [(t.shape, t.dtype) for t in copies]
        del copies
        again = [torch.empty(n, dtype=t, device="cuda") for n, t in shapes]
        for t in again:
            t.fill_(1 if t.dtype == torch.int32 else 85)
        assert cycles == 1 or not s.query(), "the stream woke up too early to show anything"
        s.synchronize()
    return result


@typed(TYPES)
def test_grouped(dtype):
    T, E, K, N = 600, 3, 136, 264
    X, W, o = torch.randn((T, K), device="cuda").to(dtype), torch.randn((E, K, N), device="cuda").to(dtype), dev([0, 99, 100, 600])
    dY = torch.randn((T, N), device="cuda").to(dtype)
    torch.cuda.synchronize()
    y = on_a_busy_stream(lambda X, W, o, s: g.sgemm_grouped(X, W, o, stream=s), X, W, o)
    assert torch.equal(y, g.sgemm_grouped(X, W, o))
    dw = on_a_busy_stream(lambda X, dY, o, s: g.sgemm_grouped_wgrad(X, dY, o, stream=s), X, dY, o)
    assert torch.equal(dw, g.sgemm_grouped_wgrad(X, dY, o))


def test_mxfp4():
    T, E, K, N = 600, 3, 160, 264
    X, W, o = torch.randn((T, K), device="cuda"), torch.randn((E, N, K), device="cuda"), dev([0, 99, 100, 600])
    a, r, b = g.sgemm_mxfp4_quantize(X, o), g.sgemm_mxfp4_quantize(X), g.sgemm_mxfp4_quantize(W)
    codes, _ = on_a_busy_stream(lambda X, o, s: g.sgemm_mxfp4_quantize(X, o, stream=s), X, o)
    assert torch.equal(codes, a[0])
    v = on_a_busy_stream(lambda c, q, o, s: g.sgemm_mxfp4_dequantize(c, q, o, stream=s), *a, o)
    assert torch.equal(v, g.sgemm_mxfp4_dequantize(*a, o))
    y = on_a_busy_stream(lambda x, xs, w, ws, o, s: g.sgemm_mxfp4_grouped(x, xs, w, ws, o, stream=s), *a, *b, o)
    assert torch.equal(y, g.sgemm_mxfp4_grouped(*a, *b, o))
    w = (b[0][0].contiguous(), b[1][0].contiguous())
    c = on_a_busy_stream(lambda x, xs, w, ws, s: g.sgemm_mxfp4(x, xs, w, ws, stream=s), *r, *w)
    assert torch.equal(c, g.sgemm_mxfp4(*r, *w))
