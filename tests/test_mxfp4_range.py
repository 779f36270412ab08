"""MXFP4 values and products near the ends of float32's range."""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from parity import TOL
from test_experts import TYPES, check, dev, typed

pytestmark = pytest.mark.gpu
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_every_scale_reads_back(dtype):
    """All 16 codes under all 256 scale bytes: exact up to 252, past float32's largest (3.4e38 < 2^128) an infinity, 255 NaN."""
    code = torch.arange(32) % 16
    codes = (code[0::2] | code[1::2] << 4).to(torch.uint8).repeat(256, 1).cuda()
    scales = torch.zeros((2, 1, 32, 4, 4), dtype=torch.uint8, device="cuda")
    r = torch.arange(256, device="cuda")
    scales[r // 128, 0, r % 32, r % 128 // 32, 0] = r.to(torch.uint8)
    got = g.sgemm_mxfp4_dequantize(codes, scales, dtype=dtype).cpu().double()
    value = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64)[code]
    want = value[None] * torch.exp2(torch.arange(256).double() - 127)[:, None]
    want = torch.where(want.abs() >= 2.0 ** 128, torch.inf * want.sign(), want)
    assert torch.equal(got[:255], want[:255])
    assert got[:253].isfinite().all() and got[253:255].isinf().any()
    assert got[255].isnan().all()


@typed(TYPES)
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("shape", [(5, 200, 1056), (300, 264, 1000)], ids=str)
@pytest.mark.parametrize("a,b", [(-100, -100), (-100, -30), (-73, -73), (-70, -70), (-60, -66), (-124, 100), (-20, -110), (59, 57), (100, 14), (-30, 125)])
def test_products(a, b, shape, grouped, dtype):
    """Rows of about 2^a times rows of about 2^b.  What a product or a sum loses below 2^-149 is 2^-149 for each 64 of the
    contraction; at the upper end the sums of magnitudes stay below 2^128."""
    M, N, K = shape
    gen = torch.Generator(device="cuda").manual_seed(1)

    def operand(rows, e):  # (codes, scales, values)
        x = torch.randn((rows, K), generator=gen, device="cuda")
        codes, scales = g.sgemm_mxfp4_quantize((x.double() * 2.0 ** e).float())
        return codes, scales, g.sgemm_mxfp4_dequantize(codes, scales, cols=K).double()

    (x, sx, vx), (w, sw, vw) = operand(M, a), operand(N, b)
    if grouped:
        o = dev([0, M // 3, M])
        x, sx = g.sgemm_mxfp4_quantize(vx.float(), o)  # (values that MXFP4 holds are returned unchanged)
        y = g.sgemm_mxfp4_grouped(x, sx, w[None].repeat(2, 1, 1), sw[None].repeat(2, 1, 1, 1, 1, 1), o, dtype=dtype)
    else:
        y = g.sgemm_mxfp4(x, sx, w, sw, dtype=dtype)
    exact, bound = vx @ vw.T, vx.abs() @ vw.abs().T
    assert bound.max() < 2.0 ** 127
    check(y, exact, bound + (K // 64 + 1) * 2.0 ** -149 / TOL)
    assert g.check_status() == 0
