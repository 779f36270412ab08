"""Products grouped by expert: forward and both gradients, against plain products in 64 bits.

Acceptance, per element: |y - exact| <= TOL * b + u * (|exact| + TOL * b) + tiny, with b = sum_k |a_k||b_k| the bound that
every entry of the library keeps in float32 (TOL = 5e-5), u the output type's unit roundoff (half its spacing at 1: 2^-8 for
bf16, 2^-11 for f16; float32's own rounding is inside TOL * b) and tiny half its smallest subnormal.  A value past the
type's largest rounds to the infinity of its sign.
"""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from parity import TOL

U = {torch.float32: 0.0, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float16: torch.finfo(torch.float16).eps / 2}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}


def typed(params):
    return pytest.mark.parametrize("dtype", params, ids=[NAMES[t] for t in params])


def check(y, exact, bound, what=""):
    assert y.shape == exact.shape, what
    lim = TOL * bound + U[y.dtype] * (exact.abs() + TOL * bound) + TINY[y.dtype]
    err = (y.double() - exact).abs()
    most = torch.finfo(y.dtype).max
    over = y.isinf() & (y.sign() == exact.sign()) & (exact.abs() * (1 + U[y.dtype]) + TOL * bound >= most)
    bad = ~(err <= lim) & ~over
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"{y[bad][0].item()} vs {exact[bad][0].item()}, allowed {lim[bad][0].item()}")


def padded(x, pad=0, shift=0):
    """x in a buffer whose rows are `pad` elements wider (NaN), begun `shift` elements in."""
    lead, cols = x.shape[:-1], x.shape[-1]
    n = x.numel() // max(cols, 1)
    store = torch.full((n * (cols + pad) + shift,), float("nan"), dtype=x.dtype, device=x.device)
    v = store[shift:].view(lead + (cols + pad,))[..., :cols]
    v.copy_(x)
    return v


def bounds_of(offsets, T):
    """The boundaries as the operators take them: clamped to [0, T], running maximum."""
    o, out = 0, []
    for i, v in enumerate(offsets):
        v = min(max(v, 0), T)
        o = v if i == 0 else max(o, v)
        out.append(o)
    return out


def operands(T, E, K, N, dtype, seed=0, transw=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn((T, K), generator=gen, device="cuda").to(dtype)
    W = torch.randn((E, N, K) if transw else (E, K, N), generator=gen, device="cuda").to(dtype)
    return X, W


def forward64(X, W, offsets, transw=False):
    o = bounds_of(offsets, X.shape[0])
    N = W.shape[1 if transw else 2]
    Y = torch.zeros((X.shape[0], N), dtype=torch.float64, device=X.device)
    B = Y.clone()
    for e in range(W.shape[0]):
        w = W[e].double().T if transw else W[e].double()
        x = X[o[e]: o[e + 1]].double()
        Y[o[e]: o[e + 1]] = x @ w
        B[o[e]: o[e + 1]] = x.abs() @ w.abs()
    return Y, B


def wgrad64(X, dY, offsets, E):
    o = bounds_of(offsets, X.shape[0])
    out = torch.zeros((E, X.shape[1], dY.shape[1]), dtype=torch.float64, device=X.device)
    B = out.clone()
    for e in range(E):
        x, d = X[o[e]: o[e + 1]].double(), dY[o[e]: o[e + 1]].double()
        out[e], B[e] = x.T @ d, x.abs().T @ d.abs()
    return out, B


def dev(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


# (T, E, K, N, offsets): one token to many, groups of none, one group, widths off every tile and every vector
SHAPES = [
    (1, 1, 1, 1, [0, 1]),
    (1, 8, 64, 128, [0, 0, 0, 1, 1, 1, 1, 1, 1]),
    (3, 2, 31, 17, [0, 1, 3]),
    (5, 4, 128, 136, [0, 0, 5, 5, 5]),
    (40, 3, 72, 264, [0, 7, 23, 40]),
    (130, 4, 200, 72, [0, 129, 129, 130, 130]),
    (257, 2, 65, 129, [0, 256, 257]),
    (600, 5, 328, 520, [0, 1, 17, 300, 300, 600]),
    (777, 3, 1025, 255, [0, 256, 512, 777]),
    (1500, 3, 256, 640, [0, 700, 701, 1500]),
    (64, 70, 96, 80, [min(i, 64) for i in range(71)]),
    (150, 8, 136, 288, [0, 0, 131, 132, 132, 140, 150, 150, 150]),
    (300, 40, 136, 256, [0] * 5 + [13 * i for i in range(23)] + [300] * 13),
]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:4])))
def test_forward(shape, transw, dtype):
    T, E, K, N, offsets = shape
    X, W = operands(T, E, K, N, dtype, 1, transw)
    exact, bound = forward64(X, W, offsets, transw)
    check(g.sgemm_grouped(X, W, dev(offsets), transw=transw), exact, bound)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (0, 8), (3, 0), (1, 5)])
@pytest.mark.parametrize("transw", [False, True])
def test_forward_strides_and_alignment(pad, shift, transw, dtype):
    T, E, K, N, offsets = 333, 3, 136, 200, [0, 100, 101, 333]
    X, W = operands(T, E, K, N, dtype, 2, transw)
    exact, bound = forward64(X, W, offsets, transw)
    out = padded(torch.zeros((T, N), dtype=dtype, device="cuda"), pad, shift)
    whole = out.untyped_storage()
    y = g.sgemm_grouped(padded(X, pad, shift), padded(W, pad, shift), dev(offsets), out, transw=transw)
    assert y is out
    check(y, exact, bound)
    store = torch.empty(0, dtype=dtype, device="cuda").set_(whole, 0, (whole.nbytes() // out.element_size(),), (1,))
    assert int(store.isnan().sum()) == shift + T * pad, "padding was written"


@pytest.mark.gpu
@typed(TYPES)
def test_forward_tensor_exact_on_integers(dtype):
    """Integers in -8..8 (int64 sums below 2^11 in f16's exact range by a short K): exact in every type but for the output's rounding."""
    T, E, K, N, offsets = 200, 3, 24, 136, [0, 3, 150, 200]
    gen = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randint(-2, 3, (T, K), generator=gen, device="cuda").to(dtype)
    W = torch.randint(-2, 3, (E, K, N), generator=gen, device="cuda").to(dtype)
    exact, _ = forward64(X, W, offsets)
    assert torch.equal(g.sgemm_grouped(X, W, dev(offsets)).double(), exact)


OFFSETS = [
    [5, 50, 60, 90],          # rows of no expert at both ends
    [0, 0, 0, 0],             # no rows at all
    [100, 100, 100, 100],     # none, all before the first
    [0, 70, 30, 100],         # a decreasing entry: an empty group
    [-7, 40, 2000000000, 5],  # out of range at both ends
    [2000000000, -5, 3, 7],   # first boundary past the end
]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("offsets", OFFSETS, ids=str)
def test_rows_of_no_expert_and_boundaries_out_of_order(offsets, dtype):
    T, E, K, N = 100, 3, 136, 264
    X, W = operands(T, E, K, N, dtype, 4)
    out = torch.full((T, N), float("nan"), dtype=dtype, device="cuda")
    exact, bound = forward64(X, W, offsets)
    check(g.sgemm_grouped(X, W, dev(offsets), out), exact, bound)
    dY = torch.randn((T, N), device="cuda").to(dtype)
    exact, bound = wgrad64(X, dY, offsets, E)
    check(g.sgemm_grouped_wgrad(X, dY, dev(offsets)), exact, bound)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_in_their_own_rows(bad, dtype):
    """Non-finite rows of a neighbouring group, of no group, and weights of another expert reach nothing else."""
    T, E, K, N, offsets = 300, 4, 72, 136, [2, 100, 101, 290, 290]
    X, W = operands(T, E, K, N, dtype, 5)
    dY = torch.randn((T, N), device="cuda").to(dtype)
    exact, bound = forward64(X, W, offsets)
    dexact, dbound = wgrad64(X, dY, offsets, E)
    X, W, dY = X.clone(), W.clone(), dY.clone()
    for t in (0, 1, 100, 295, 299):  # rows of no group, and the whole of group 1
        X[t], dY[t] = bad, bad
    W[3] = bad  # an expert without rows
    y = g.sgemm_grouped(X, W, dev(offsets))
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[100] = False
    check(y[keep], exact[keep], bound[keep])
    assert not y[100].isfinite().any()
    dw = g.sgemm_grouped_wgrad(X, dY, dev(offsets))
    for e in (0, 2, 3):
        check(dw[e], dexact[e], dbound[e], f"expert {e}")
    assert not dw[1].isfinite().any()
    # one bad element: its own row of the output only
    X, W = operands(T, E, K, N, dtype, 5)
    X[50, 7] = bad
    y = g.sgemm_grouped(X, W, dev(offsets))
    keep[100], keep[50] = True, False
    check(y[keep], exact[keep], bound[keep])
    assert not y[50].isfinite().any()


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:4])))
def test_wgrad(shape, out32, dtype):
    T, E, K, N, offsets = shape
    X, _ = operands(T, E, K, N, dtype, 6)
    dY = torch.randn((T, N), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda").to(dtype)
    exact, bound = wgrad64(X, dY, offsets, E)
    dw = g.sgemm_grouped_wgrad(X, dY, dev(offsets), dtype=torch.float32 if out32 else None)
    assert dw.dtype == (torch.float32 if out32 else dtype)
    check(dw, exact, bound)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (1, 5)])
def test_wgrad_strides_and_alignment(pad, shift, dtype):
    T, E, K, N, offsets = 333, 3, 136, 200, [0, 100, 101, 333]
    X, _ = operands(T, E, K, N, dtype, 8)
    dY = torch.randn((T, N), device="cuda").to(dtype)
    exact, bound = wgrad64(X, dY, offsets, E)
    out = padded(torch.zeros((E, K, N), dtype=dtype, device="cuda"), pad, shift)
    check(g.sgemm_grouped_wgrad(padded(X, pad, shift), padded(dY, pad, shift), dev(offsets), out), exact, bound)


@pytest.mark.gpu
@typed(TYPES)
def test_gradients_against_differences(dtype):
    """The product is linear in each operand: a central difference of L = sum(Y * R) along one element, computed by the
    forward operator itself, is the gradient up to rounding.  Step 1 on operands of a few bits, so that in every type
    each product and sum is exact and the two must be equal."""
    T, E, K, N, offsets = 60, 3, 40, 48, [0, 20, 21, 60]
    gen = torch.Generator(device="cuda").manual_seed(9)

    def ints(*shape):
        return torch.randint(-2, 3, shape, generator=gen, device="cuda").to(dtype)

    X, W, R = ints(T, K), ints(E, K, N), ints(T, N)
    o = dev(offsets)
    dX = g.sgemm_grouped(R, W, o, transw=True)
    dW = g.sgemm_grouped_wgrad(X, R, o)

    def loss(x, w):
        return (g.sgemm_grouped(x, w, o).double() * R.double()).sum()

    for t, k in ((0, 0), (19, 39), (20, 3), (59, 17)):
        hi, lo = X.clone(), X.clone()
        hi[t, k] += 1
        lo[t, k] -= 1
        assert ((loss(hi, W) - loss(lo, W)) / 2).item() == dX[t, k].item()
    for e, k, n in ((0, 0, 0), (1, 39, 47), (2, 5, 31)):
        hi, lo = W.clone(), W.clone()
        hi[e, k, n] += 1
        lo[e, k, n] -= 1
        assert ((loss(X, hi) - loss(X, lo)) / 2).item() == dW[e, k, n].item()


@pytest.mark.gpu
@typed(TYPES)
def test_transposed_weights_gradient(dtype):
    """Weights stored (E, N, K): swapping X and dY gives their gradient."""
    T, E, K, N, offsets = 90, 2, 40, 72, [0, 33, 90]
    X, _ = operands(T, E, K, N, dtype, 10)
    dY = torch.randn((T, N), device="cuda").to(dtype)
    exact, bound = wgrad64(X, dY, offsets, E)
    check(g.sgemm_grouped_wgrad(dY, X, dev(offsets)), exact.mT, bound.mT)


@pytest.mark.gpu
def test_other_streams_and_graphs():
    T, E, K, N, offsets = 200, 4, 256, 384, [0, 10, 10, 150, 200]
    X, W = operands(T, E, K, N, torch.bfloat16, 11)
    exact, bound = forward64(X, W, offsets)
    o = dev(offsets)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = g.sgemm_grouped(X, W, o, stream=s)
    s.synchronize()
    check(y, exact, bound)
    # recorded once, replayed on other rows and other groups
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((E, K, N), dtype=torch.float32, device="cuda")
    dY = torch.randn((T, N), device="cuda").to(torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.sgemm_grouped(X, W, o, out)
        g.sgemm_grouped_wgrad(X, dY, o, dw)
    for seed, new in ((12, [0, 0, 199, 200, 200]), (13, [0, 50, 100, 150, 200])):
        X.copy_(operands(T, E, K, N, torch.bfloat16, seed)[0])
        o.copy_(dev(new))
        graph.replay()
        torch.cuda.synchronize()
        check(out, *forward64(X, W, new))
        check(dw, *wgrad64(X, dY, new, E))


@pytest.mark.gpu
@typed(TYPES)
def test_results_do_not_depend_on_timing(dtype):
    T, E, K, N = 500, 6, 1032, 264
    offsets = [0, 1, 2, 100, 360, 360, 500]
    X, W = operands(T, E, K, N, dtype, 14)
    dY = torch.randn((T, N), device="cuda").to(dtype)
    o = dev(offsets)
    y, dw = g.sgemm_grouped(X, W, o), g.sgemm_grouped_wgrad(X, dY, o)
    for _ in range(5):
        assert torch.equal(g.sgemm_grouped(X, W, o), y)
        assert torch.equal(g.sgemm_grouped_wgrad(X, dY, o), dw)


@pytest.mark.gpu
@typed(TYPES)
def test_empty_sizes(dtype):
    X, W = operands(4, 2, 8, 16, dtype)
    o = dev([0, 2, 4])
    assert g.sgemm_grouped(X[:0], W, dev([0, 0, 0])).shape == (0, 16)
    assert g.sgemm_grouped(X, W[:, :, :0], o).shape == (4, 0)
    assert torch.equal(g.sgemm_grouped(X[:, :0], W[:, :0], o), torch.zeros((4, 16), dtype=dtype, device="cuda"))
    assert torch.equal(g.sgemm_grouped(X, W[:0], dev([0])), torch.zeros((4, 16), dtype=dtype, device="cuda"))
    assert torch.equal(g.sgemm_grouped_wgrad(X[:0], W[0, :0], dev([0, 0, 0])),
                       torch.zeros((2, 8, 16), dtype=dtype, device="cuda"))
    assert g.sgemm_grouped_wgrad(X, X, dev([0])).shape == (0, 8, 8)


@pytest.mark.gpu
def test_binding_refuses():
    X, W = operands(4, 2, 8, 16, torch.bfloat16)
    o = dev([0, 2, 4])
    with pytest.raises(TypeError):
        g.sgemm_grouped(X.cpu(), W, o)
    with pytest.raises(TypeError):
        g.sgemm_grouped(X, W.float(), o)
    with pytest.raises(TypeError):
        g.sgemm_grouped(X.double(), W.double(), o)
    with pytest.raises(TypeError):
        g.sgemm_grouped(X, W, o.long())
    with pytest.raises(ValueError):
        g.sgemm_grouped(X, W, o[:2])
    with pytest.raises(ValueError):
        g.sgemm_grouped(X, W, o, transw=True)
    with pytest.raises(ValueError):
        g.sgemm_grouped(X, W[0], o)
    with pytest.raises(ValueError):
        g.sgemm_grouped(X.T.contiguous().T, W, o)
    with pytest.raises(ValueError):
        g.sgemm_grouped(X[:1].expand(4, 8), W, o)
    with pytest.raises(ValueError):
        g.sgemm_grouped(X, W, o, torch.empty((4, 16), device="cuda"))
    with pytest.raises(g.SgemmError):
        g.sgemm_grouped(X, W, o, W[0, :4])  # the output in the weights
    with pytest.raises(ValueError):
        g.sgemm_grouped_wgrad(X, X[:3], o)
    with pytest.raises(TypeError):
        g.sgemm_grouped_wgrad(X, X, o, dtype=torch.float16)


FAKE_X, FAKE_W, FAKE_O, FAKE_Y = 0x10000000, 0x20000000, 0x30000000, 0x40000000  # never dereferenced


@pytest.mark.parametrize("change", [
    {"type": 3}, {"type": -1}, {"transw": 2}, {"T": -1}, {"E": -1}, {"N": -1}, {"K": -1}, {"X": 0}, {"W": 0}, {"o": 0},
    {"Y": 0}, {"ldx": 7}, {"ldw": 15}, {"sw": 127}, {"ldy": 15}, {"X": FAKE_X + 1}, {"W": FAKE_W + 1}, {"o": FAKE_O + 2},
    {"Y": FAKE_Y + 1}, {"Y": FAKE_X + 16}, {"Y": FAKE_W + 16}, {"ldx": 1 << 60}, {"sw": 1 << 61}, {"T": (1 << 30) + 1},
], ids=str)
def test_invalid_arguments_rejected_on_host(change):
    from dense_fp32_gemm_f32_gb300 import _lib

    a = {"type": 1, "transw": 0, "T": 4, "E": 2, "N": 16, "K": 8, "X": FAKE_X, "ldx": 8, "W": FAKE_W, "ldw": 16, "sw": 128,
         "o": FAKE_O, "Y": FAKE_Y, "ldy": 16} | change
    lib = _lib.load()
    assert lib.sgemm_grouped(*a.values(), None) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    {"type": 3}, {"out": 2}, {"out": 5}, {"T": -1}, {"E": -1}, {"K": -1}, {"N": -1}, {"X": 0}, {"dY": 0}, {"o": 0}, {"dW": 0},
    {"ldx": 7}, {"lddy": 15}, {"lddw": 15}, {"sdw": 127}, {"dW": FAKE_X}, {"dW": FAKE_W}, {"dW": FAKE_Y + 1},
], ids=str)
def test_invalid_gradient_arguments_rejected_on_host(change):
    from dense_fp32_gemm_f32_gb300 import _lib

    a = {"type": 1, "out": 1, "T": 4, "E": 2, "K": 8, "N": 16, "X": FAKE_X, "ldx": 8, "dY": FAKE_W, "lddy": 16, "o": FAKE_O,
         "dW": FAKE_Y, "lddw": 16, "sdw": 128} | change
    lib = _lib.load()
    assert lib.sgemm_grouped_wgrad(*a.values(), None) == _lib.ERR_INVALID_ARG


def test_header_states_which_entry_points_allocate():
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "sgemm_experts.h")).read()
    listed = [re.search(r"^\s*\*\s*" + tag + r":\s*([\w ]+)$", text, flags=re.M).group(1).split()
              for tag in ("EXPERTS-ALLOCATING", "EXPERTS-NON-ALLOCATING")]
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = re.findall(r"^\s*int\s+(sgemm_\w+)\s*\(", code, flags=re.M)
    assert sorted(listed[0] + listed[1]) == sorted(declared)


@pytest.fixture(autouse=True)
def no_wait_gave_up(request):
    """After every GPU test: no kernel abandoned a bounded wait."""
    yield
    if request.node.get_closest_marker("gpu"):
        assert g.check_status() == 0


# Sizes at which the rule on tiles takes each of them: many tiles of 256 columns, few of 128, single CTAs; float32
# with few rows an expert, its contraction split over CTAs.
TILES = [
    (3000, 4, 136, 1024, [0, 700, 1500, 2999, 3000]),
    (800, 4, 264, 520, [0, 200, 401, 600, 800]),
    (200, 3, 1200, 392, [0, 60, 61, 200]),
    (5, 1, 2100, 300, [0, 5]),
    (12, 2, 4100, 136, [0, 3, 12]),
    (100, 4, 2052, 520, [0, 0, 9, 60, 100]),
]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("shape", TILES, ids=lambda s: "x".join(map(str, s[:4])))
def test_forward_every_tile(shape, transw, dtype):
    T, E, K, N, offsets = shape
    X, W = operands(T, E, K, N, dtype, 21, transw)
    exact, bound = forward64(X, W, offsets, transw)
    check(g.sgemm_grouped(X, W, dev(offsets), transw=transw), exact, bound)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("shape", [(300, 4, 520, 1100, [0, 64, 128, 299, 300]), (2000, 2, 256, 384, [0, 1990, 2000])],
                         ids=lambda s: "x".join(map(str, s[:4])))
def test_wgrad_every_tile(shape, dtype):
    T, E, K, N, offsets = shape
    X, _ = operands(T, E, K, N, dtype, 22)
    dY = torch.randn((T, N), device="cuda").to(dtype)
    check(g.sgemm_grouped_wgrad(X, dY, dev(offsets)), *wgrad64(X, dY, offsets, E))


@pytest.mark.gpu
@typed([torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [1, 2, 4, 8])
def test_output_rows_of_every_alignment(pad, dtype):
    """Outputs whose rows are aligned to 2, 4, 8 and 16 bytes, and whose widths end at every part of a store; nothing past
    a row's end is written."""
    T, E, K, offsets = 150, 2, 72, [0, 70, 150]
    for N in (33, 34, 36, 40, 64, 129):
        X, W = operands(T, E, K, N, dtype, 23)
        out = padded(torch.zeros((T, N), dtype=dtype, device="cuda"), pad)
        check(g.sgemm_grouped(X, W, dev(offsets), out), *forward64(X, W, offsets))
        dY = torch.randn((T, N), device="cuda").to(dtype)
        dw = padded(torch.zeros((E, K, N), dtype=dtype, device="cuda"), pad)
        check(g.sgemm_grouped_wgrad(X, dY, dev(offsets), dw), *wgrad64(X, dY, offsets, E))
        for v in (out, dw):
            store = torch.empty(0, dtype=dtype, device="cuda").set_(v.untyped_storage(), 0, (v.untyped_storage().nbytes() // v.element_size(),), (1,))
            assert int(store.isnan().sum()) == v.numel() // N * pad, N


@pytest.mark.gpu
def test_outputs_past_2_to_the_31_elements():
    T, N, K, offsets = 70000, 40000, 16, [0, 69000, 70000]
    X, W = operands(T, 2, K, N, torch.bfloat16, 24)
    y = g.sgemm_grouped(X, W, dev(offsets))
    assert y.numel() > 2 ** 31
    for r in (slice(0, 3), slice(53686, 53690), slice(68998, 69003), slice(69990, 70000)):
        at = [min(max(o - r.start, 0), r.stop - r.start) for o in offsets]
        check(y[r], *forward64(X[r], W, at))
    del y, W
    torch.cuda.empty_cache()
    T, K, N = 20, 30000, 30000
    X = torch.randn((T, K), device="cuda").to(torch.bfloat16)
    dY = torch.randn((T, N), device="cuda").to(torch.bfloat16)
    dw = g.sgemm_grouped_wgrad(X, dY, dev([0, 5, 5, 20]))
    assert dw.numel() > 2 ** 31
    for rows in (slice(0, 2), slice(29990, 30000)):
        check(dw[:, rows], *wgrad64(X[:, rows], dY, [0, 5, 5, 20], 3))
    del dw
    torch.cuda.empty_cache()


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("transw", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 600, 130, [0, 1]), (9, 6, 3000, 136, [0, 0, 2, 2, 9, 9, 9]), (90, 1, 5000, 264, [0, 88]),
                                   (4, 40, 2090, 72, [0, 1, 1, 2, 4] + [4] * 36)], ids=lambda s: "x".join(map(str, s[:4])))
def test_contraction_split_over_ctas(shape, transw, dtype):
    """Few tiles and a long contraction: a cluster of CTAs adds up its parts."""
    T, E, K, N, offsets = shape
    X, W = operands(T, E, K, N, dtype, 25, transw)
    exact, bound = forward64(X, W, offsets, transw)
    y = g.sgemm_grouped(X, W, dev(offsets), transw=transw)
    check(y, exact, bound)
    assert torch.equal(y, g.sgemm_grouped(X, W, dev(offsets), transw=transw))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,K,N", [(torch.float32, 256, 384), (torch.float32, 255, 130), (torch.float16, 131, 130)], ids=str)
def test_graphs_with_operand_copies(dtype, K, N):
    """Calls that take a copy of their operands from the pool, recorded and replayed on other rows and groups."""
    T, E = 200, 3
    X, W = operands(T, E, K, N, dtype, 26)
    dY = torch.randn((T, N), device="cuda").to(dtype)
    o = dev([0, 60, 61, 200])
    g.sgemm_grouped(X, W, o)  # (the library's first call on a device is made outside a capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = g.sgemm_grouped(X, W, o)
        dw = g.sgemm_grouped_wgrad(X, dY, o)
    for seed, new in ((27, [0, 0, 150, 200]), (28, [7, 100, 199, 199])):
        X.copy_(operands(T, E, K, N, dtype, seed)[0])
        o.copy_(dev(new))
        graph.replay()
        torch.cuda.synchronize()
        check(y, *forward64(X, W, new))
        check(dw, *wgrad64(X, dY, new, E))


@pytest.mark.gpu
def test_concurrent_streams():
    """Calls of every kind in flight on four streams at once."""
    T, E, K, N, offsets = 700, 4, 264, 520, [0, 100, 350, 351, 700]
    o = dev(offsets)
    sets = []
    for i, dtype in enumerate((torch.float32, torch.bfloat16, torch.float16, torch.float32)):
        X, W = operands(T, E, K, N, dtype, 30 + i)
        sets.append((X, W, torch.randn((T, N), device="cuda").to(dtype), torch.cuda.Stream()))
    torch.cuda.synchronize()
    results = []
    for _ in range(3):
        for X, W, dY, s in sets:
            results.append((X, W, dY, g.sgemm_grouped(X, W, o, stream=s), g.sgemm_grouped_wgrad(X, dY, o, stream=s)))
    torch.cuda.synchronize()
    for X, W, dY, y, dw in results:
        check(y, *forward64(X, W, offsets))
        check(dw, *wgrad64(X, dY, offsets, E))


@pytest.mark.gpu
@typed(TYPES)
def test_many_tiles_of_ragged_groups(dtype):
    """Many rounds of tiles over the GPU, of unequal groups."""
    T, E, K, N = 5000, 8, 72, 5000
    offsets = [0, 3, 1500, 1500, 2100, 2101, 3000, 4900, 4990]
    X, W = operands(T, E, K, N, dtype, 40)
    check(g.sgemm_grouped(X, W, dev(offsets)), *forward64(X, W, offsets))
    dY = torch.randn((T, 1300), device="cuda").to(dtype)
    X = torch.randn((T, 1500), device="cuda").to(dtype)
    dw = g.sgemm_grouped_wgrad(X, dY, dev(offsets * 2)[: E + 1])
    check(dw, *wgrad64(X, dY, offsets, E))
    o = sorted(offsets * 3)[: 25]
    dw = g.sgemm_grouped_wgrad(X, dY, dev(o))
    check(dw, *wgrad64(X, dY, o, 24))


@pytest.mark.gpu
@pytest.mark.parametrize("exponent", [-100, -118, -124, -130, 100])
def test_float32_magnitudes(exponent):
    """Operands near the ends of float32's range: the parts hold each to within half of 2^-133, so a row's error grows by
    2^-134 sum |w| at most; everything else is relative."""
    T, E, K, N, offsets = 100, 2, 256, 136, [0, 50, 100]
    X, W = operands(T, E, K, N, torch.float32, 50)
    X = (X.double() * 2.0 ** exponent).float()
    if exponent > 0:
        W = (W.double() * 2.0 ** -exponent).float()
    exact, bound = forward64(X, W, offsets)
    granule, _ = forward64(torch.full_like(X, 2.0 ** -134), W.abs(), offsets)
    err = (g.sgemm_grouped(X, W, dev(offsets)).double() - exact).abs()
    if exponent > 0:
        granule = granule + forward64(X.abs(), torch.full_like(W, 2.0 ** -134), offsets)[0]
    assert (err <= TOL * bound + granule + 2.0 ** -149).all(), (err / bound).max().item()
    few = g.sgemm_grouped(X[:8], W, dev([0, 4, 8])).double()  # (no parts)
    exact, bound = forward64(X[:8], W, [0, 4, 8])
    assert ((few - exact).abs() <= TOL * bound + K * 2.0 ** -149).all()


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("shape", [(1500, 3, 72, 8704, [0, 3, 900, 1490]), (2000, 2, 40, 4200, [0, 1999, 2000]), (90, 3, 72, 6300, [0, 30, 31, 90])],
                         ids=lambda s: "x".join(map(str, s[:4])))
def test_forward_wide_features(shape, dtype):
    """More feature tiles than a band of the tile order holds, the last band part full, and rows of several tiles."""
    T, E, K, N, offsets = shape
    X, W = operands(T, E, K, N, dtype, 60)
    exact, bound = forward64(X, W, offsets)
    out = torch.full((T, N), float("nan"), dtype=dtype, device="cuda")
    check(g.sgemm_grouped(X, W, dev(offsets), out=out), exact, bound)
