"""MXFP4: quantisation against its definition on the CPU, bit for bit, and the products against sums in 64 bits."""
import math

import numpy as np
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import TYPES, bounds_of, check, dev, padded, typed

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def nearest(u):
    """Code of the magnitude u >= 0: nearest of the grid's, ties to the even code, at most 6."""
    best = 0
    for c in range(1, 8):
        d, b = abs(u - GRID[c]), abs(u - GRID[best])
        if d < b or (d == b and c % 2 == 0):
            best = c
    return best


def quantize_row(row):
    """(codes, scale bytes) of one row, from the definition, in Python's own arithmetic."""
    codes, scales = [], []
    for k in range(0, len(row), 32):
        b = [float(v) for v in row[k: k + 32]]
        if not all(math.isfinite(v) for v in b):
            codes += [None] * 32
            scales.append(255)
            continue
        m = max(abs(v) for v in b)
        s = max(math.frexp(m)[1] - 1 - 2, -127) if m else -127
        scales.append(s + 127)
        codes += [nearest(abs(v) * 2.0 ** -s) | (8 if math.copysign(1, v) < 0 else 0) for v in b] + [0] * (32 - len(b))
    return codes, scales


def unpack(codes):
    c = codes.cpu().numpy()
    out = np.empty(c.shape[:-1] + (2 * c.shape[-1],), dtype=np.int64)
    out[..., 0::2], out[..., 1::2] = c & 15, c >> 4
    return out


def scale_at(scales, r, b):
    """Scale byte of row r, block b from the documented place in memory."""
    kq = scales.shape[-4]
    flat = scales.cpu().numpy().reshape(scales.shape[:-5] + (-1,))
    return flat[..., ((r // 128) * kq + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4]


def special_rows(K, dtype, seed=0):
    """Rows with what a quantiser gets wrong: ties, ranges' ends, zeros, signs of zero, subnormals, infinities, NaN."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((12, K), generator=gen) * torch.exp2(torch.randint(-20, 20, (12, 1), generator=gen).float())
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, 0.0, -0.0, -0.25, -2.5, -5.0, -7.75])
    x[1] = ties.repeat(K // 16 + 1)[:K] * 2.0 ** -3
    x[2] = 0
    x[3] = -0.0
    x[4] = torch.finfo(dtype).max
    x[5] = torch.finfo(dtype).smallest_normal * torch.rand(K, generator=gen)
    x[6] = torch.finfo(dtype).tiny * 2.0 ** -5
    x[7, K // 2] = float("inf")
    x[8, K - 1] = float("nan")
    x[9, 0] = -float("inf")
    x[10] = torch.exp2(torch.arange(K).float() % 12 - 9)
    x[11, K // 3:] = 0
    return x.to(dtype)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("K", [1, 31, 32, 33, 96, 160, 1024, 1500])
def test_quantize_bits(K, dtype):
    x = special_rows(K, dtype, K)
    codes, scales = g.sgemm_mxfp4_quantize(x.cuda())
    kb = (K + 31) // 32
    assert codes.shape == (12, 16 * kb) and scales.shape == (1, (K + 127) // 128, 32, 4, 4)
    got = unpack(codes)
    for r in range(12):
        want, ws = quantize_row(x[r].tolist())
        assert [scale_at(scales, r, b) for b in range(kb)] == ws, r
        assert all(w is None or w == c for w, c in zip(want, got[r])), r
        for b in range(kb, 4 * scales.shape[1]):
            assert scale_at(scales, r, b) == 0
    # the values read back
    v = g.sgemm_mxfp4_dequantize(codes, scales, cols=K)
    for r in range(12):
        want, ws = quantize_row(x[r].tolist())
        for k in range(K):
            if want[k] is None:
                assert math.isnan(v[r, k])
            else:
                assert v[r, k].item() == (-1 if want[k] & 8 else 1) * GRID[want[k] & 7] * 2.0 ** (ws[k // 32] - 127), (r, k)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (1, 5)])
def test_quantize_batches_strides_and_alignment(pad, shift, dtype):
    x = torch.randn((3, 140, 200), device="cuda").to(dtype)
    codes, scales = g.sgemm_mxfp4_quantize(padded(x, pad, shift))
    assert scales.shape == (3, 2, 2, 32, 4, 4)
    for e in range(3):
        c, s = g.sgemm_mxfp4_quantize(x[e].contiguous())
        assert torch.equal(codes[e], c)
        # (rows past the matrix hold anything)
        rows = torch.arange(140)
        for b in range(7):
            assert np.array_equal(scale_at(scales[e], rows.numpy(), b), scale_at(s, rows.numpy(), b))
    for out in (torch.float32, torch.bfloat16, torch.float16):
        y = padded(torch.zeros((3, 140, 200), dtype=out, device="cuda"), pad, shift)
        g.sgemm_mxfp4_dequantize(codes, scales, cols=200, out=y)
        assert torch.equal(y.float(), g.sgemm_mxfp4_dequantize(codes, scales, cols=200).to(out).float())


@pytest.mark.gpu
def test_quantize_exact_values_come_back():
    """Values that MXFP4 holds are returned unchanged."""
    gen = torch.Generator().manual_seed(0)
    v = torch.tensor(GRID)[torch.randint(0, 8, (50, 256), generator=gen)] * (torch.randint(0, 2, (50, 256), generator=gen) * 2 - 1)
    v[:, ::32] = 6.0
    v *= torch.exp2(torch.randint(-100, 100, (50, 8, 1), generator=gen).float()).expand(50, 8, 32).reshape(50, 256)
    codes, scales = g.sgemm_mxfp4_quantize(v.cuda())
    assert torch.equal(g.sgemm_mxfp4_dequantize(codes, scales).cpu(), v)
    assert torch.equal(g.sgemm_mxfp4_dequantize(codes, scales, dtype=torch.bfloat16).cpu().float(), v)


GROUPS = [(300, [0, 1, 1, 130, 259, 300]), (70, [5, 10, 40, 60]), (10, [0, 0, 0]), (200, [0, 150, 20, 900]),
          (90, [min(2 * i, 90) for i in range(60)])]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("T,offsets", GROUPS, ids=str)
def test_quantize_grouped(T, offsets, dtype):
    """Grouped rows: the same codes, every expert's scales in blocks of its own; rows of none read back as zeros."""
    x = torch.randn((T, 300), device="cuda").to(dtype)
    o = dev(offsets)
    codes, scales = g.sgemm_mxfp4_quantize(x, o)
    plain, pscales = g.sgemm_mxfp4_quantize(x)
    assert torch.equal(codes, plain)
    b = bounds_of(offsets, T)
    block = 0
    for e in range(len(offsets) - 1):
        n = b[e + 1] - b[e]
        r = np.arange(n)
        for q in range(10):
            assert np.array_equal(scale_at(scales, 128 * block + r, q), scale_at(pscales, b[e] + r, q)), e
        block += (n + 127) // 128
    assert block <= scales.shape[0]
    y = g.sgemm_mxfp4_dequantize(codes, scales, o, cols=300)
    want = g.sgemm_mxfp4_dequantize(plain, pscales, cols=300)
    want[: b[0]] = 0
    want[b[-1]:] = 0
    assert torch.equal(y, want)


def random_mxfp4(shape, seed, spread=6):
    """Random codes and scales of (..., rows, K), and their values in 64 bits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=gen, device="cuda") * torch.exp2(
        torch.randint(-spread, spread, shape[:-1] + (1,), generator=gen, device="cuda").float())
    codes, scales = g.sgemm_mxfp4_quantize(x)
    return codes, scales, g.sgemm_mxfp4_dequantize(codes, scales, cols=shape[-1]).double()


PRODUCTS = [(1, 1, 1), (1, 128, 64), (5, 200, 96), (16, 136, 1056), (128, 128, 128), (129, 257, 65), (300, 520, 1000),
            (256, 256, 4096), (700, 384, 544),
            (33, 130, 160), (64, 136, 288), (65, 128, 96), (193, 264, 352), (385, 72, 192)]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, dtype):
    a, sa, va = random_mxfp4((M, K), 1)
    b, sb, vb = random_mxfp4((N, K), 2)
    check(g.sgemm_mxfp4(a, sa, b, sb, dtype=dtype), va @ vb.T, va.abs() @ vb.abs().T)
    out = padded(torch.zeros((M, N), dtype=dtype, device="cuda"), 3, 1)
    check(g.sgemm_mxfp4(a, sa, b, sb, out), va @ vb.T, va.abs() @ vb.abs().T)


@pytest.mark.gpu
def test_product_exact_on_small_sums():
    """Codes with equal scales: every product a multiple of 1/4 below 2^6, sums exact in float32."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    v = torch.tensor(GRID, device="cuda")
    x = v[torch.randint(0, 8, (150, 512), generator=gen, device="cuda")]
    w = -v[torch.randint(0, 8, (260, 512), generator=gen, device="cuda")]
    x[:, ::32] = 6
    w[:, ::32] = -6
    (a, sa), (b, sb) = g.sgemm_mxfp4_quantize(x), g.sgemm_mxfp4_quantize(w)
    assert torch.equal(g.sgemm_mxfp4(a, sa, b, sb, dtype=torch.float32).double(), x.double() @ w.double().T)


@pytest.mark.gpu
def test_product_non_finite_rows_and_unused_scales():
    """A block that stands for NaN reaches its own row only; scales of rows beyond the matrix reach nothing."""
    x = torch.randn((40, 200), device="cuda")
    x[7, 100] = float("nan")
    w = torch.randn((50, 200), device="cuda")
    w[9, 3] = float("inf")
    (a, sa), (b, sb) = g.sgemm_mxfp4_quantize(x), g.sgemm_mxfp4_quantize(w)
    va, vb = g.sgemm_mxfp4_dequantize(a, sa, cols=200).double(), g.sgemm_mxfp4_dequantize(b, sb, cols=200).double()
    for s, rows in ((sa, 40), (sb, 50)):  # (32 rows x 4: row r is at [r % 32, r / 32])
        for r in range(rows, 128):
            s[0, :, r % 32, r // 32] = 255
    c = g.sgemm_mxfp4(a, sa, b, sb, dtype=torch.float32)
    keep = torch.ones((40, 50), dtype=torch.bool, device="cuda")
    keep[7], keep[:, 9] = False, False
    assert c[~keep].isnan().all()
    va, vb = va.nan_to_num(), vb.nan_to_num()
    check(c[keep], (va @ vb.T)[keep], (va.abs() @ vb.abs().T)[keep])


EXPERTS = [(1, 4, 128, 96, [0, 0, 1, 1, 1]), (20, 3, 200, 1024, [0, 3, 3, 20]), (300, 5, 264, 416, [0, 1, 1, 130, 259, 300]),
           (70, 3, 136, 65, [5, 10, 40, 60]), (200, 3, 128, 256, [0, 150, 20, 900]), (100, 2, 128, 64, [0, 0, 0]),
           (800, 2, 640, 1152, [0, 300, 800]),
           (150, 8, 136, 288, [0, 0, 131, 132, 132, 140, 150, 150, 150]), (500, 3, 200, 96, [0, 65, 258, 500]), (80, 40, 72, 160, [2 * i for i in range(41)])]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("T,E,N,K,offsets", EXPERTS, ids=str)
def test_grouped_product(T, E, N, K, offsets, dtype):
    w, sw, vw = random_mxfp4((E, N, K), 4)
    x = torch.randn((T, K), device="cuda")
    o = dev(offsets)
    a, sa = g.sgemm_mxfp4_quantize(x, o)
    va = g.sgemm_mxfp4_dequantize(a, sa, o, cols=K).double()
    b = bounds_of(offsets, T)
    exact = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    bound = exact.clone()
    for e in range(E):
        exact[b[e]: b[e + 1]] = va[b[e]: b[e + 1]] @ vw[e].T
        bound[b[e]: b[e + 1]] = va[b[e]: b[e + 1]].abs() @ vw[e].abs().T
    out = torch.full((T, N), float("nan"), dtype=dtype, device="cuda")
    y = g.sgemm_mxfp4_grouped(a, sa, w, sw, o, out)
    check(y, exact, bound)
    assert torch.equal(y, g.sgemm_mxfp4_grouped(a, sa, w, sw, o, dtype=dtype))


@pytest.mark.gpu
def test_streams_and_graphs():
    x, w = torch.randn((30, 256), device="cuda"), torch.randn((2, 136, 256), device="cuda")
    o = dev([0, 11, 30])
    wc, ws = g.sgemm_mxfp4_quantize(w)

    def layer(stream=None):
        a, sa = g.sgemm_mxfp4_quantize(x, o, stream=stream)
        return g.sgemm_mxfp4_grouped(a, sa, wc, ws, o, dtype=torch.float32, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = layer(s)
    s.synchronize()
    assert torch.equal(y, layer())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    x.normal_()
    o.copy_(dev([0, 30, 30]))
    graph.replay()
    assert torch.equal(out, layer())


@pytest.mark.gpu
def test_empty_sizes():
    e = torch.empty((0, 64), device="cuda")
    codes, scales = g.sgemm_mxfp4_quantize(e)
    assert codes.shape == (0, 32) and scales.shape == (0, 1, 32, 4, 4)
    assert g.sgemm_mxfp4_dequantize(codes, scales).shape == (0, 64)
    b, sb = g.sgemm_mxfp4_quantize(torch.ones((3, 64), device="cuda"))
    assert g.sgemm_mxfp4(codes, scales, b, sb).shape == (0, 3)
    z, sz = g.sgemm_mxfp4_quantize(torch.empty((3, 0), device="cuda"))
    assert torch.equal(g.sgemm_mxfp4(z, sz, z, sz, dtype=torch.float32), torch.zeros((3, 3), device="cuda"))


@pytest.mark.gpu
def test_binding_refuses():
    x = torch.randn((4, 64), device="cuda")
    a, sa = g.sgemm_mxfp4_quantize(x)
    with pytest.raises(TypeError):
        g.sgemm_mxfp4_quantize(x.double())
    with pytest.raises(TypeError):
        g.sgemm_mxfp4_quantize(x.cpu())
    with pytest.raises(ValueError):
        g.sgemm_mxfp4_quantize(x.T)
    with pytest.raises(ValueError):
        g.sgemm_mxfp4_quantize(x[None], dev([0, 4]))
    with pytest.raises(ValueError):
        g.sgemm_mxfp4_quantize(x, codes=torch.empty((4, 16), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        g.sgemm_mxfp4_dequantize(a, sa, cols=65)
    with pytest.raises(ValueError):
        g.sgemm_mxfp4_dequantize(a, sa[:, :, :16], cols=64)
    with pytest.raises(TypeError):
        g.sgemm_mxfp4(x, sa, a, sa)
    with pytest.raises(ValueError):
        g.sgemm_mxfp4(a[:, :16].contiguous(), sa, a, sa)
    with pytest.raises(TypeError):
        g.sgemm_mxfp4(a, sa, a, sa, dtype=torch.float64)
    with pytest.raises(ValueError):
        g.sgemm_mxfp4_grouped(a, sa, a[None], sa[None], dev([0, 1, 4]))


FAKE = {"X": 0x10000000, "xs": 0x20000000, "W": 0x30000000, "ws": 0x40000000, "o": 0x50000000, "Y": 0x60000000}


@pytest.mark.parametrize("change", [
    {"type": 3}, {"T": -1}, {"E": -1}, {"N": -1}, {"K": -1}, {"X": 0}, {"xs": 0}, {"W": 0}, {"ws": 0}, {"o": 0}, {"Y": 0},
    {"X": 0x10000008}, {"xs": 0x20000008}, {"W": 0x30000001}, {"ws": 0x40000004}, {"ldy": 15}, {"Y": 0x60000001},
    {"Y": 0x10000010}, {"Y": 0x40000010},
], ids=str)
def test_invalid_arguments_rejected_on_host(change):
    from dense_fp32_gemm_f32_gb300 import _lib

    a = {"type": 1, "T": 4, "E": 2, "N": 16, "K": 64} | FAKE | {"ldy": 16} | change
    lib = _lib.load()
    assert lib.sgemm_mxfp4_grouped(*a.values(), None) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    {"type": 3}, {"batch": -1}, {"rows": -1}, {"K": -1}, {"X": 0}, {"X": 0x10000002}, {"ldx": 63}, {"sx": 3}, {"E": 1},
    {"E": -1}, {"o": 0x50000000}, {"codes": 0}, {"codes": 0x30000008}, {"scales": 0}, {"scales": 0x10000000},
], ids=str)
def test_invalid_quantize_arguments_rejected_on_host(change):
    from dense_fp32_gemm_f32_gb300 import _lib

    a = {"type": 0, "batch": 2, "rows": 4, "K": 64, "X": 0x10000000, "ldx": 64, "sx": 256, "E": 0, "o": None,
         "codes": 0x30000000, "scales": 0x40000000} | change
    lib = _lib.load()
    assert lib.sgemm_mxfp4_quantize(*a.values(), None) == _lib.ERR_INVALID_ARG


@pytest.fixture(autouse=True)
def no_wait_gave_up(request):
    """After every GPU test: no kernel abandoned a bounded wait."""
    yield
    if request.node.get_closest_marker("gpu"):
        assert g.check_status() == 0


@pytest.mark.gpu
def test_arrays_past_2_to_the_31_elements():
    x = torch.randn((40, 60000), device="cuda").to(torch.bfloat16).repeat(1000, 1)
    assert x.numel() > 2 ** 31
    codes, scales = g.sgemm_mxfp4_quantize(x)
    few, fs = g.sgemm_mxfp4_quantize(x[:128].contiguous())
    assert torch.equal(codes[-40:], few[:40])
    y = g.sgemm_mxfp4_dequantize(codes, scales, dtype=torch.bfloat16)
    assert torch.equal(y[-40:], g.sgemm_mxfp4_dequantize(few, fs, dtype=torch.bfloat16)[:40])
    del x, y, codes, scales
    torch.cuda.empty_cache()
    a, sa, va = random_mxfp4((60000, 64), 5)
    b, sb, vb = random_mxfp4((40000, 64), 6)
    c = g.sgemm_mxfp4(a, sa, b, sb)
    assert c.numel() > 2 ** 31
    for r in (slice(0, 2), slice(53680, 53690), slice(59995, 60000)):
        check(c[r], va[r] @ vb.T, va[r].abs() @ vb.abs().T)
    del c
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [1, 2, 4, 8])
def test_product_output_rows_of_every_alignment(pad):
    for N in (33, 34, 36, 40, 193):
        a, sa, va = random_mxfp4((70, 96), 7)
        b, sb, vb = random_mxfp4((N, 96), 8)
        out = padded(torch.zeros((70, N), dtype=torch.float16, device="cuda"), pad)
        check(g.sgemm_mxfp4(a, sa, b, sb, out), va @ vb.T, va.abs() @ vb.abs().T)
        store = torch.empty(0, dtype=torch.float16, device="cuda").set_(out.untyped_storage(), 0, (out.untyped_storage().nbytes() // 2,), (1,))
        assert int(store.isnan().sum()) == 70 * pad


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("T,E,N,K,offsets", [(3, 1, 200, 5000, [0, 3]), (40, 1, 130, 2080, [0, 40]), (64, 2, 392, 9000, [0, 1, 64]),
                                             (9, 6, 136, 4128, [0, 0, 2, 2, 9, 9, 9]), (70, 2, 128, 8192, [3, 68, 68])], ids=str)
def test_contraction_split_over_ctas(T, E, N, K, offsets, dtype):
    """Few tiles and a long contraction: a cluster of CTAs adds up its parts."""
    w, sw, vw = random_mxfp4((E, N, K), 9)
    x = torch.randn((T, K), device="cuda")
    o = dev(offsets)
    a, sa = g.sgemm_mxfp4_quantize(x, o)
    va = g.sgemm_mxfp4_dequantize(a, sa, o, cols=K).double()
    b = bounds_of(offsets, T)
    exact = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    bound = exact.clone()
    for e in range(E):
        exact[b[e]: b[e + 1]] = va[b[e]: b[e + 1]] @ vw[e].T
        bound[b[e]: b[e + 1]] = va[b[e]: b[e + 1]].abs() @ vw[e].abs().T
    y = g.sgemm_mxfp4_grouped(a, sa, w, sw, o, dtype=dtype)
    check(y, exact, bound)
    assert torch.equal(y, g.sgemm_mxfp4_grouped(a, sa, w, sw, o, dtype=dtype))
    if E == 1:
        a, sa = g.sgemm_mxfp4_quantize(x)
        assert torch.equal(y, g.sgemm_mxfp4(a, sa, w[0], sw[0], dtype=dtype))


@pytest.mark.gpu
def test_many_tiles_of_ragged_groups():
    """Many rounds of tiles over the GPU, of unequal groups."""
    T, E, N, K, offsets = 5000, 6, 5000, 160, [0, 3, 1500, 2100, 2101, 4000, 4990]
    w, sw, vw = random_mxfp4((E, N, K), 10)
    x = torch.randn((T, K), device="cuda")
    o = dev(offsets)
    a, sa = g.sgemm_mxfp4_quantize(x, o)
    va = g.sgemm_mxfp4_dequantize(a, sa, o, cols=K).double()
    exact = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    bound = exact.clone()
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        exact[r], bound[r] = va[r] @ vw[e].T, va[r].abs() @ vw[e].abs().T
    check(g.sgemm_mxfp4_grouped(a, sa, w, sw, o), exact, bound)
