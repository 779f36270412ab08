"""Long contractions whose products have one sign, and sums that begin with their largest product: what an accumulator cuts
or rounds away at each step adds up instead of cancelling.

The acceptance is the one of test_experts.py, the bound that the header states: 5e-5 sum |a||b|, and the output's rounding.
Where it comes from, for a contraction of K <= 2^17:
* tensor cores, 16-bit operands: an instruction cuts each of its 16 products 2^-25 below the largest magnitude in it and the
  sum 2^-23 below, 6e-7 of sum |a||b|; 64 of them go into one accumulator, 3.9e-5, and each accumulator is added to a
  float32 register, 2^-24 each: K / 1024 * 2^-24 = 7.6e-6.
* float32 in parts: 32 instructions of the leading products into one accumulator, 1.9e-5; K / 512 * 2 additions, 3.1e-5 at
  2^17, 1.1e-5 for the 45000 here.
* float32, few rows: 512 additions in a row at 2^-24, 3.1e-5, and K / 4096 more.
* MXFP4: an instruction of 64 cuts the sum 2^-23 below; 256 of them, 3.1e-5; K / 16384 additions.
"""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import TYPES, bounds_of, check, dev, forward64, typed, wgrad64


def positive(shape, kind, gen, dtype):
    """Positive values, the contraction along dimension -2: "even" in [1/2, 1); "peak" with a first row 2^9 times as large
    (2^18 in a product of two such operands)."""
    x = torch.rand(shape, generator=gen, device="cuda") * 0.5 + 0.5
    if kind == "peak":
        x *= 2.0 ** -6
        x[..., 0, :] *= 2.0 ** 9
    return x.to(dtype)


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    assert g.check_status() == 0


pytestmark = pytest.mark.gpu


@typed(TYPES)
@pytest.mark.parametrize("kind", ["even", "peak"])
@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("K,N,E,T,offsets", [(72, 136, 3, 45000, [5, 15, 44990, 45000]), (1032, 1500, 2, 9000, [0, 8990, 9000])], ids=["narrow", "wide"])
def test_wgrad(K, N, E, T, offsets, kind, out32, dtype):
    gen = torch.Generator(device="cuda").manual_seed(1)
    X, dY = positive((T, K), "even", gen, dtype), positive((T, N), "even", gen, dtype)
    for e in range(E):
        if offsets[e] < offsets[e + 1]:
            rows = slice(offsets[e], offsets[e + 1])
            X[rows], dY[rows] = (positive((rows.stop - rows.start, n), kind, gen, dtype) for n in (K, N))
    dw = g.sgemm_grouped_wgrad(X, dY, dev(offsets), dtype=torch.float32 if out32 else None)
    check(dw, *wgrad64(X, dY, offsets, E))


# (rows, columns, contraction): a contraction shared by a cluster, single CTAs, pairs with both widths of tile
FORWARD = [(3, 200, 45000), (40, 10300, 9000), (150, 400, 45000), (2000, 2000, 9000)]


@typed(TYPES)
@pytest.mark.parametrize("kind", ["even", "peak"])
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("T,N,K", FORWARD)
def test_forward(T, N, K, transw, kind, dtype):
    gen = torch.Generator(device="cuda").manual_seed(2)
    X, W = positive((K, T), kind, gen, dtype).T.contiguous(), positive((1, K, N), kind, gen, dtype)
    if transw:
        W = W.mT.contiguous()
    offsets = [0, T]
    check(g.sgemm_grouped(X, W, dev(offsets), transw=transw), *forward64(X, W, offsets, transw))


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


# (rows, columns, contraction): a contraction shared by a cluster (one accumulator a CTA, several), single CTAs, pairs
PRODUCTS = [(3, 200, 100000), (3, 200, 262144), (20, 200, 140000), (40, 10300, 20000), (300, 200, 131072), (900, 700, 40000)]


@typed([torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["peak", "blocks"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_mxfp4(M, N, K, kind, dtype):
    """"peak": a first block of 32 whose products are 2^20 times as large; "blocks": blocks of magnitudes within 2^12."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def operand(rows):
        x = torch.rand((rows, K), generator=gen, device="cuda") * 0.9 + 0.1
        if kind == "peak":
            x[:, :32] *= 2.0 ** 10
        else:
            s = torch.exp2(torch.randint(-6, 7, (rows, (K + 31) // 32, 1), generator=gen, device="cuda").float())
            x *= s.expand(-1, -1, 32).reshape(rows, -1)[:, :K]
        codes, scales = g.sgemm_mxfp4_quantize(x)
        return codes, scales, g.sgemm_mxfp4_dequantize(codes, scales, cols=K)

    (a, sa, va), (b, sb, vb) = operand(M), operand(N)
    c = g.sgemm_mxfp4(a, sa, b, sb, dtype=dtype)
    vb = vb[-512:].double()  # (the last columns)
    exact = va.double() @ vb.T
    check(c[:, -512:], exact, exact.abs())


@pytest.mark.parametrize("T,offsets", [(500, [3, 200, 201, 500]), (30, [0, 0, 20, 29])], ids=str)
def test_mxfp4_grouped(T, offsets):
    """Groups of unequal sizes, a contraction past one accumulator's that ends inside a slice."""
    K, N, E = 33000, 264, 3
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.rand((T, K), generator=gen, device="cuda") * torch.exp2(
        torch.randint(-6, 7, (T, 1), generator=gen, device="cuda").float())
    w = torch.rand((E, N, K), generator=gen, device="cuda")
    o = dev(offsets)
    a, sa = g.sgemm_mxfp4_quantize(x, o)
    b, sb = g.sgemm_mxfp4_quantize(w)
    va, vb = g.sgemm_mxfp4_dequantize(a, sa, o, cols=K).double(), g.sgemm_mxfp4_dequantize(b, sb, cols=K).double()
    bounds = bounds_of(offsets, T)
    exact = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    for e in range(E):
        exact[bounds[e]: bounds[e + 1]] = va[bounds[e]: bounds[e + 1]] @ vb[e].T
    out = torch.full((T, N), float("nan"), device="cuda")
    check(g.sgemm_mxfp4_grouped(a, sa, b, sb, o, out), exact, exact.abs())
