"""Orthogonalised updates against the same steps in 64 bits.

Tolerances, in the 2-norm relative to the result's.  Rounding errors made at a step are multiplied at most like the values
themselves by the steps after it: an error in the direction of singular values that the remaining steps raise by g is raised
by g, while the result's norm is that of all directions brought near 1.
bf16: three roundings of f16 operands a step (X, O, P), each within 2^-12 of the element and 2^-12 / sqrt(3) in the mean, in
the parts of the polynomial that they stand in, |b| s^2 and 2 c s^4 with s <= 1.2: below 7 and 9 at most, and small for all
but the last three steps (singular values are small before).  Nine of them, were they all at their largest at once, come to
8 sqrt(9) 2^-12 / sqrt(3) = 2^-8.2; 2^-8 is what the header promises.
float32 and f16: operands of 22 bits, 2^-11 times as much, and sums in float32, cut to 24 bits every 16 of the contraction
(32 times 2^-24 in an accumulator at most, 2^-19): 2^-18.
Then the output's rounding, half a step of its type relative to each element.
"""
import math

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from dense_fp32_gemm_f32_gb300 import _lib
from test_experts import padded, typed

TYPES = [torch.float32, torch.bfloat16, torch.float16]
LIMIT = {torch.float32: 2.0 ** -18, torch.bfloat16: 2.0 ** -8 + 2.0 ** -8, torch.float16: 2.0 ** -18 + 2.0 ** -11}
QUINTIC = (3.4445, -4.7750, 2.0315)


def ortho64(G, steps=5, coefficients=QUINTIC, eps=1e-7):
    a, b, c = coefficients
    X = G.double()
    X = X / (X.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    for _ in range(steps):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.mT if tall else X


def check(y, exact, factor=1.0):
    assert y.shape == exact.shape
    off = (y.double() - exact).flatten(-2).norm(dim=-1) / exact.flatten(-2).norm(dim=-1)
    assert (off <= factor * LIMIT[y.dtype]).all(), off.max().item()
    assert g.check_status() == 0


def update(E, M, N, dtype, seed=0, rank=0, size=1e-3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    G = torch.randn((E, M, N), generator=gen, device="cuda")
    if rank:
        u, v = (torch.randn(s, generator=gen, device="cuda") for s in ((E, M, rank), (E, rank, N)))
        G = 0.2 * G + u @ v / math.sqrt(rank)
    return (G * size).to(dtype)


# ------------------------------------------------------------------ refusals, on the CPU

A, B, C = 0x10000000, 0x20000000, 0x30000000  # never dereferenced


@pytest.mark.parametrize("change", [
    dict(type=3), dict(E=-1), dict(M=-1), dict(N=-1), dict(G=0), dict(out=0), dict(G=A + 1), dict(ldg=31), dict(ldo=31), dict(sg=400),
    dict(so=100), dict(out=A + 64), dict(steps=0), dict(steps=65), dict(a=math.nan), dict(b=math.inf), dict(eps=-1.0), dict(eps=math.nan),
    dict(eps=math.inf), dict(a=4.0, b=0.0, c=0.0), dict(a=1.5, b=0.0, c=0.0), dict(c=30.0), dict(a=0.0, b=-100.0, c=100.0),
    dict(M=2 ** 24, N=2 ** 24, ldg=2 ** 24, ldo=2 ** 24, sg=2 ** 48, so=2 ** 48, out=1 << 55),
    # a workspace that is missing, too small, not aligned, or G's or the result's
    dict(M=200, N=256, ldg=256, ldo=256, sg=51200, so=51200), dict(M=200, N=256, ldg=256, ldo=256, sg=51200, so=51200, workspace=C, bytes=10 ** 6),
    dict(M=200, N=256, ldg=256, ldo=256, sg=51200, so=51200, workspace=C + 128, bytes=10 ** 8),
    dict(M=200, N=256, ldg=256, ldo=256, sg=51200, so=51200, workspace=A + 4096, bytes=10 ** 8),
    dict(M=200, N=256, ldg=256, ldo=256, sg=51200, so=51200, workspace=B - 4096, bytes=10 ** 8)], ids=str)
def test_refusals(change):
    p = dict(type=1, E=2, M=16, N=32, G=A, ldg=32, sg=512, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, out=B, ldo=32, so=512, workspace=0, bytes=0,
             stream=None)
    p.update(change)
    assert _lib.load().sgemm_orthogonalize(*p.values()) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("coefficients", [QUINTIC, (2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (1.0, 0.0, 0.0)])
def test_usual_polynomials_are_taken(coefficients):
    """(Of no matrices: nothing is launched.)"""
    assert _lib.load().sgemm_orthogonalize(1, 0, 16, 32, 0, 32, 512, 64, *coefficients, 0.0, 0, 32, 512, 0, 0, None) == _lib.OK


def test_binding_refuses_cpu_tensors():
    with pytest.raises(TypeError):
        g.sgemm_orthogonalize(torch.zeros(4, 4))


def test_workspace():
    """What a call takes: nothing for short sides, the planes of X twice and of A and B once, each of two f16 values an element;
    no size for what is refused."""
    size = _lib.load().sgemm_orthogonalize_workspace
    assert size(1, 8, 128, 2048, 5) == size(0, 1, 2000, 100, 5) == size(1, 0, 500, 500, 5) == size(1, 2, 500, 0, 5) == 0
    least = 2 * 2 * 8 * (2 * 2048 * 4096 + 2 * 2048 * 2048)
    assert least <= size(1, 8, 2048, 4096, 5) <= 1.01 * least
    assert size(1, 8, 2048, 4096, 1) <= least - 2 * 2 * 8 * 2048 * 4096 * 0.99
    assert size(3, 1, 500, 500, 5) == size(1, -1, 500, 500, 5) == size(1, 1, 500, 500, 0) == size(1, 1, 2 ** 25, 2 ** 25, 5) == -1


def test_header_states_that_it_does_not_allocate():
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sgemm_ortho.h")
    assert "ORTHO-NON-ALLOCATING: sgemm_orthogonalize sgemm_orthogonalize_workspace\n" in open(path).read()


# ------------------------------------------------------------------ results

SHAPES = [(1, 1, 1), (1, 1, 7), (2, 9, 1), (1, 2, 3), (3, 16, 16), (1, 31, 64), (2, 64, 31), (1, 65, 130), (1, 128, 128), (2, 129, 127),
          (5, 96, 200), (1, 200, 1000), (1, 1000, 130), (1, 257, 255), (2, 300, 520), (1, 513, 511), (2, 700, 640), (1, 1100, 1300)]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("rank", [0, 3])
@pytest.mark.parametrize("E,M,N", SHAPES)
def test_orthogonalize(E, M, N, rank, dtype):
    G = update(E, M, N, dtype, seed=M + N, rank=rank)
    check(g.sgemm_orthogonalize(G), ortho64(G))


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("E,M,N", [(6, 1024, 1536), (7, 1536, 1000), (40, 260, 256), (3, 8192, 264), (1, 512, 5000)])
def test_orthogonalize_many_tiles(E, M, N, dtype):
    G = update(E, M, N, dtype, seed=1, rank=8)
    check(g.sgemm_orthogonalize(G), ortho64(G))


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("E,M,N", [(1, 128, 129), (2, 100, 256), (1, 128, 257), (3, 385, 17), (1, 90, 640), (2, 128, 1024), (1, 1025, 127),
                                   (1, 60, 2049), (2, 3000, 128), (1, 128, 4096), (1, 33, 3841), (1, 128, 4097), (40, 64, 300), (170, 9, 20)])
def test_short_sides(E, M, N, dtype):
    """A short side of up to 128, in clusters of one to sixteen CTAs, and a long one past what those hold."""
    G = update(E, M, N, dtype, seed=M + N, rank=2)
    y = g.sgemm_orthogonalize(G)
    check(y, ortho64(G))
    assert torch.equal(y, g.sgemm_orthogonalize(G))


@pytest.mark.gpu
@typed(TYPES)
def test_one_matrix_without_a_batch(dtype):
    G = update(1, 130, 70, dtype, seed=2)
    y = g.sgemm_orthogonalize(G[0])
    assert y.shape == (130, 70)
    assert torch.equal(y, g.sgemm_orthogonalize(G)[0])


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (0, 8), (3, 0), (1, 5)])
@pytest.mark.parametrize("M,N", [(72, 136), (136, 72), (130, 300), (300, 130)])
def test_strides_and_alignment(M, N, pad, shift, dtype):
    G = update(3, M, N, dtype, seed=3)
    out = padded(torch.zeros_like(G), pad, shift)
    whole = out.untyped_storage()
    y = g.sgemm_orthogonalize(padded(G, pad, shift), out)
    assert y is out
    check(y, ortho64(G))
    store = torch.empty(0, dtype=dtype, device="cuda").set_(whole, 0, (whole.nbytes() // out.element_size(),), (1,))
    assert int(store.isnan().sum()) == shift + 3 * M * pad, "padding was written"


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("steps,coefficients", [(1, QUINTIC), (2, QUINTIC), (3, (2.0, -1.5, 0.5)), (12, (2.0, -1.5, 0.5)), (6, (1.5, -0.5, 0.0)),
                                                (4, (1.0, 0.0, 0.0))])
def test_steps_and_polynomials(steps, coefficients, dtype):
    G = update(2, 150, 260, dtype, seed=4)
    check(g.sgemm_orthogonalize(G, steps=steps, coefficients=coefficients), ortho64(G, steps, coefficients))


@pytest.mark.gpu
@typed(TYPES)
def test_converged_result_is_orthogonal(dtype):
    """A polynomial that converges to 1: U V^T of the singular value decomposition, and stays there.  G's singular values are
    within a factor of 4, so 12 steps leave less than 2^-30 of the way."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    u, _ = torch.linalg.qr(torch.randn((100, 60), generator=gen, device="cuda", dtype=torch.float64))
    v, _ = torch.linalg.qr(torch.randn((60, 60), generator=gen, device="cuda", dtype=torch.float64))
    G = ((u * torch.linspace(1, 4, 60, device="cuda", dtype=torch.float64)) @ v.T).to(dtype)
    U, _, V = torch.linalg.svd(G.double(), full_matrices=False)
    check(g.sgemm_orthogonalize(G, steps=12, coefficients=(2.0, -1.5, 0.5))[None], (U @ V)[None])


@pytest.mark.gpu
@typed([torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e-12, 1.0, 1e15, 1e36])
def test_sizes_from_end_to_end_of_the_type(size, dtype):
    """Squares that float32 cannot hold; the result does not depend on the size (eps = 0)."""
    G = update(2, 70, 90, torch.float32, seed=6, size=1.0)
    G = (G * size).to(dtype)
    check(g.sgemm_orthogonalize(G, eps=0.0), ortho64(G, eps=0.0))


@pytest.mark.gpu
def test_smallest_numbers():
    G = update(1, 40, 30, torch.float32, seed=7, size=1.0) * 2.0 ** -100 * 2.0 ** -45
    assert (G != 0).any()
    check(g.sgemm_orthogonalize(G, eps=0.0), ortho64(G, eps=0.0))


@pytest.mark.gpu
@typed(TYPES)
def test_eps_zeros_and_sparse_matrices(dtype):
    G = update(4, 66, 130, dtype, seed=8, size=1.0)
    G[1] = 0
    G[2, 5:] = 0          # five rows
    G[3] = 0
    G[3, 7, 11] = -3      # one element
    y = g.sgemm_orthogonalize(G)
    assert (y[1] == 0).all()
    check(y[[0, 2, 3]], ortho64(G[[0, 2, 3]]))
    check(g.sgemm_orthogonalize(G[:1], eps=50.0), ortho64(G[:1], eps=50.0))


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("M,N", [(66, 130), (130, 66), (300, 600), (20, 1500)])
def test_a_non_finite_element_stays_in_its_matrix(M, N, bad, dtype):
    G = update(3, M, N, dtype, seed=9)
    G[1, M // 2, N // 3] = bad
    y = g.sgemm_orthogonalize(G)
    assert not y[1].isfinite().any()
    check(y[[0, 2]], ortho64(G[[0, 2]]))


@pytest.mark.gpu
@typed(TYPES)
def test_nothing_to_do(dtype):
    for shape in ((0, 4, 4), (2, 0, 4), (2, 4, 0), (0, 5)):
        assert g.sgemm_orthogonalize(torch.zeros(shape, dtype=dtype, device="cuda")).shape == shape


@pytest.mark.gpu
def test_binding_checks():
    G = torch.zeros((2, 8, 12), device="cuda")
    for call in (lambda: g.sgemm_orthogonalize(G[0, 0]), lambda: g.sgemm_orthogonalize(G.mT), lambda: g.sgemm_orthogonalize(G, G[:1].clone()),
                 lambda: g.sgemm_orthogonalize(G[:1].expand(2, 8, 12).mT)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        g.sgemm_orthogonalize(G.double())
    for call in (lambda: g.sgemm_orthogonalize(G, G), lambda: g.sgemm_orthogonalize(G, steps=0), lambda: g.sgemm_orthogonalize(G, coefficients=(9, 9, 9)),
                 lambda: g.sgemm_orthogonalize(G[:1].expand(2, 8, 12))):
        with pytest.raises(g.SgemmError):
            call()


@pytest.mark.gpu
@typed(TYPES)
def test_results_do_not_depend_on_timing(dtype):
    G = update(3, 520, 300, dtype, seed=10)
    y = g.sgemm_orthogonalize(G)
    for _ in range(3):
        assert torch.equal(g.sgemm_orthogonalize(G), y)
    for e in range(3):  # nor on the other matrices
        assert torch.equal(g.sgemm_orthogonalize(G[e]), y[e])


@pytest.mark.gpu
@typed([torch.float32, torch.bfloat16])
def test_streams_and_recorded_calls(dtype):
    """Calls on four streams at once, and two graphs replayed at the same time: each has its own workspace."""
    shapes = [(2, 300, 200), (1, 64, 64), (1, 130, 700), (3, 257, 256)]
    G = [update(*s, dtype, seed=20 + i) for i, s in enumerate(shapes)]
    want = [g.sgemm_orthogonalize(x) for x in G]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    got = [[g.sgemm_orthogonalize(x, stream=s) for x, s in zip(G, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for ys in got for y, w in zip(ys, want))
    graphs, out = [], []
    for x in G[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out.append(g.sgemm_orthogonalize(x))
        graphs.append(graph)
    for seed in range(2):
        for i, x in enumerate(G[:2]):
            x.copy_(update(*shapes[i], dtype, seed=30 + 2 * seed + i))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(G, out):
            assert torch.equal(g.sgemm_orthogonalize(x), y)
    assert g.check_status() == 0


@pytest.mark.gpu
def test_a_workspace_of_anything():
    """What the scratch held before has no part in the result (NaN, counters that are not zero)."""
    G = update(2, 300, 520, torch.bfloat16, seed=35)
    want, lib = g.sgemm_orthogonalize(G), _lib.load()
    n = lib.sgemm_orthogonalize_workspace(_lib.TYPE_BF16, 2, 300, 520, 5)
    for fill in (0, 0xFF, 0x7F):
        scratch, out = torch.full((n,), fill, dtype=torch.uint8, device="cuda"), torch.empty_like(G)
        rc = lib.sgemm_orthogonalize(_lib.TYPE_BF16, 2, 300, 520, G.data_ptr(), 520, 300 * 520, 5, *QUINTIC, 1e-7, out.data_ptr(), 520,
                                     300 * 520, scratch.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert rc == _lib.OK and torch.equal(out, want)


@pytest.mark.gpu
def test_the_weight_gradients_of_experts():
    """As used: the gradients of grouped products, an expert without rows among them."""
    T, E, K, N = 400, 4, 136, 264
    gen = torch.Generator(device="cuda").manual_seed(40)
    X, dY = (torch.randn((T, w), generator=gen, device="cuda").to(torch.bfloat16) for w in (K, N))
    offsets = torch.tensor([0, 150, 150, 390, 400], dtype=torch.int32, device="cuda")
    dW = g.sgemm_grouped_wgrad(X, dY, offsets)
    y = g.sgemm_orthogonalize(dW)
    assert (y[1] == 0).all()
    check(y[[0, 2, 3]], ortho64(dW[[0, 2, 3]]))
