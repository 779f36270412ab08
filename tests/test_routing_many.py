"""Many tokens: the same choices, token by token, as a few at a time, which test_routing.py compares with 64 bits."""
import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from test_experts import typed
from test_routing import TYPES, check_route, randn

pytestmark = pytest.mark.gpu

INF = float("inf")
HOW = [dict(), dict(renormalize=True, scale=2.5), dict(score="sigmoid", bias=1, renormalize=True), dict(bias=1), dict(score="sigmoid", bias=0),
       dict(groups=2, top_groups=1, group_best=2), dict(groups=4, top_groups=2, bias=1), dict(groups=8, top_groups=4, group_best=2, bias=1, score="sigmoid"),
       dict(groups=8, top_groups=3, score="sigmoid"), dict(groups=4, top_groups=3, group_best=2, bias=0), dict(groups=32, top_groups=5, group_best=2, bias=1)]


def some_logits(T, E, dtype):
    """Random ones, quarters, near ones, rows of one value, rows and experts out of service, NaN and infinities."""
    l = randn(T, E, seed=T + E)
    l[::5] = (4 * l[::5]).round() / 4
    l[1::7] = 1 + 1e-6 * l[1::7]
    l[2::31] = -1.5
    l[3::37] = -INF
    l[4::41, 1:] = -INF
    l[5::43, ::3] = -INF
    l[6::47, E // 2] = float("nan")
    l[8::53, E // 3] = INF
    l[9::59] *= 1e4
    return l.to(dtype)


@typed(TYPES)
@pytest.mark.parametrize("how", HOW, ids=str)
@pytest.mark.parametrize("T, E, k", [(513, 8, 1), (700, 16, 2), (1030, 40, 3), (521, 64, 8), (2000, 96, 5), (999, 128, 8), (3000, 160, 7), (1500, 256, 8),
                                     (20011, 32, 4), (40007, 256, 6)])
def test_as_a_few_at_a_time(T, E, k, how, dtype):
    how = dict(how)
    if E % how.get("groups", 1):
        how.update(groups=2, top_groups=1)
    if "bias" in how:
        how["bias"] = 0.1 * randn(E, seed=3) if how["bias"] else torch.full((E,), 0.25, device="cuda")
    logits = some_logits(T, E, dtype)
    r = g.sgemm_route(logits, k, **how)
    for t0 in {0, T // 3, T - 500}:
        few = g.sgemm_route(logits[t0:t0 + 500], k, **how)
        assert torch.equal(r.experts[t0:t0 + 500], few.experts)
        a, b = r.weights[t0:t0 + 500], few.weights
        assert torch.equal(a.isfinite(), b.isfinite())
        a, b = a.nan_to_num(0, 0, 0), b.nan_to_num(0, 0, 0)
        assert ((a - b).abs() <= 2.0 ** -17 * b.abs().amax(-1, keepdim=True)).all()
    # the places, from all choices
    e = r.experts.flatten().long()
    order = torch.argsort(torch.where(e < 0, E, e), stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(r.slots.flatten(), torch.where(e < 0, -1, slots).int())
    counts = torch.bincount(e[e >= 0], minlength=E)
    assert r.offsets.tolist() == [0] + torch.cumsum(counts, 0).tolist()
    assert g.check_status() == 0


@typed(TYPES)
@pytest.mark.parametrize("how", [dict(), dict(score="sigmoid", bias=1, groups=8, top_groups=4, group_best=2, renormalize=True), dict(bias=1)], ids=str)
@pytest.mark.parametrize("E, k", [(64, 6), (256, 8)])
def test_many_against_64_bits(E, k, how, dtype):
    how = dict(how)
    if "bias" in how:
        how["bias"] = 0.1 * randn(E, seed=3)
    logits = randn(600, E, seed=4, dtype=dtype)
    check_route(g.sgemm_route(logits, k, **how), logits, k, **how)


@pytest.mark.parametrize("pad, shift", [(3, 1), (8, 0), (1, 0)])
@typed(TYPES)
def test_rows_apart(pad, shift, dtype):
    logits = randn(900, 256, seed=5, dtype=dtype)
    view = torch.full((900, 256 + pad), 1e4, dtype=dtype, device="cuda")[:, shift:shift + 256]
    view.copy_(logits)
    for a, b in zip(g.sgemm_route(view, 8), g.sgemm_route(logits, 8)):
        assert torch.equal(a, b)


SIZES = [(5000, 256, 8, dict(score="sigmoid", bias=1, groups=8, top_groups=4, group_best=2)), (300, 64, 6, dict()), (70000, 32, 2, dict(bias=1))]


def case(T, E, how, seed):
    how = dict(how)
    if "bias" in how:
        how["bias"] = 0.1 * randn(E, seed=3)
    return randn(T, E, seed=seed, dtype=torch.bfloat16), how


@pytest.mark.parametrize("T, E, k, how", SIZES, ids=str)
def test_many_recorded_calls(T, E, k, how):
    """Two graphs on two streams at once, replayed with other logits."""
    graphs = []
    for seed in (1, 2):
        logits, kw = case(T, E, how, seed)
        g.sgemm_route(logits, k, **kw)
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            r = g.sgemm_route(logits, k, **kw)
        graphs.append((graph, stream, logits, kw, r))
    for again in range(3):
        for i, (graph, stream, logits, kw, r) in enumerate(graphs):
            logits.copy_(case(T, E, how, 10 * again + i)[0])
        torch.cuda.synchronize()
        for graph, stream, *_ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, logits, kw, r in graphs:
            for a, b in zip(r, g.sgemm_route(logits, k, **kw)):
                assert torch.equal(a, b)
    assert g.check_status() == 0


@pytest.mark.parametrize("T, E, k, how", SIZES, ids=str)
def test_many_calls_at_once(T, E, k, how):
    """On four streams, each over other logits; every result is that of the call alone."""
    cases = [case(T, E, how, seed) for seed in range(4)]
    alone = [g.sgemm_route(logits, k, **kw) for logits, kw in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    results = [[g.sgemm_route(logits, k, stream=s, **kw) for (logits, kw), s in zip(cases, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for some in results:
        for r, want in zip(some, alone):
            assert all(torch.equal(a, b) for a, b in zip(r, want))
    assert g.check_status() == 0
