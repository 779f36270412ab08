"""Routing, spreading and combining against their definitions in 64 bits.

Tolerances.  Whole numbers (experts, boundaries, places) have to be equal.  u is the output type's unit roundoff, half its
spacing at 1, and v = 2^-24 that of the sums in float32.
Weights: within 2^-18 of the token's largest, as the header says (exp and the softmax's sum: see the kernel).
Combined rows: k products of one rounding each, added in order: (k + 1) v sum |w||y|, then u |exact|.
Gradients of the weights: a thread adds H / 32 products at most (and a vector of 8), then 5 shuffles and 8 partial sums:
(H / 32 + 24) v sum |d||y|.  Gradients of the logits: every factor is within 2^-19 relative for the logits used here
(|l - max| <= 20: 20 v for exp, 30 v for the sums, less than 12 further roundings), so 2^-18 scale s (|d| + sum s |d|), then u.
"""
import math

import pytest
import torch

import dense_fp32_gemm_f32_gb300 as g
from dense_fp32_gemm_f32_gb300 import _lib
from test_experts import TINY, padded, typed

TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {t: torch.finfo(t).eps / 2 for t in TYPES}
INF, NAN = math.inf, math.nan


# ------------------------------------------------------------------ definitions


def scores64(l, score):
    l = l.double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    top = l.max(-1, keepdim=True).values
    x = torch.exp(l - torch.where(top == -INF, 0.0, top))
    return x / x.sum(-1, keepdim=True).clamp(min=1e-300)


def route64(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_best=1, renormalize=False, scale=1.0):
    """One token after another, in Python's own numbers."""
    l = logits.double().cpu()
    s = scores64(l, score)
    c = s if bias is None else s + bias.double().cpu()
    T, E = l.shape
    top_groups = groups if top_groups is None else top_groups
    experts, weights = torch.full((T, k), -1, dtype=torch.int32), torch.zeros((T, k), dtype=torch.float64)
    by = c if bias is not None or (groups > 1 and group_best == 2) else l  # (the scores' order is the logits')
    for t in range(T):
        open_ = [e for e in range(E) if l[t, e] != -INF and c[t, e] != -INF]
        if groups > 1:
            size, value = E // groups, []
            for q in range(groups):
                best = sorted((by[t, e].item() for e in open_ if e // size == q), reverse=True)[:group_best]
                if best:
                    value.append((-sum(best), q))
            kept = {q for _, q in sorted(value)[:top_groups]}
            open_ = [e for e in open_ if e // size in kept]
        chosen = sorted(open_, key=lambda e: (-by[t, e].item(), e))[:k]
        w = s[t, chosen]
        if renormalize and chosen:
            w = torch.softmax(l[t, chosen], 0) if score == "softmax" else torch.softmax(torch.nn.functional.logsigmoid(l[t, chosen]), 0)
        experts[t, : len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        weights[t, : len(chosen)] = scale * w
    return experts, weights


def places64(experts, E):
    flat, slots, offsets = experts.flatten().tolist(), [], [0] * (E + 1)
    for e in flat:
        if e >= 0:
            offsets[e + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    at = list(offsets)
    for e in flat:
        slots.append(at[e] if e >= 0 else -1)
        if e >= 0:
            at[e] += 1
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(slots, dtype=torch.int32).view(experts.shape)


def check_route(r, logits, k, **how):
    experts, weights = route64(logits, k, **how)
    assert torch.equal(r.experts.cpu(), experts), (r.experts.cpu() != experts).nonzero()[:4]
    most = weights.abs().amax(-1, keepdim=True)
    assert ((r.weights.double().cpu() - weights).abs() <= 2.0 ** -18 * most).all()
    offsets, slots = places64(experts, logits.shape[1])
    assert torch.equal(r.offsets.cpu(), offsets) and torch.equal(r.slots.cpu(), slots)
    assert g.check_status() == 0


def randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# ------------------------------------------------------------------ refusals, on the CPU

A, B, C, D, F, H = (0x10000000 * i for i in range(1, 7))  # never dereferenced


def route_args(**change):
    a = dict(type=1, score=0, T=8, E=16, k=2, logits=A, ld=16, bias=None, groups=1, top=1, best=1, renorm=0, scale=1.0, experts=B,
             weights=C, offsets=D, slots=F, stream=None)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change", [
    dict(type=3), dict(score=2), dict(T=-1), dict(E=0), dict(E=1025, ld=1025), dict(k=0), dict(k=17), dict(k=33, E=64, ld=64),
    dict(ld=15), dict(groups=0), dict(groups=3), dict(groups=4, top=5), dict(groups=4, top=0), dict(best=0), dict(best=3),
    dict(renorm=2), dict(logits=0), dict(logits=A + 1), dict(experts=0), dict(weights=C + 2), dict(offsets=0), dict(slots=0),
    dict(experts=A), dict(slots=B + 8), dict(bias=A + 2), dict(offsets=C), dict(bias=C + 8), dict(T=2 ** 30, k=16),
    dict(groups=64, E=64, ld=64)], ids=str)
def test_route_refuses(change):
    assert _lib.load().sgemm_route(*route_args(**change)) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(type=-1), dict(score=-1), dict(T=-1), dict(k=0), dict(k=17), dict(ld=15), dict(experts=0), dict(dweights=0), dict(out=0),
    dict(ldd=15), dict(out=A + 16), dict(out=B), dict(renorm=-1), dict(out=H + 1)], ids=str)
def test_route_grad_refuses(change):
    a = dict(type=1, score=0, T=8, E=16, k=2, logits=A, ld=16, experts=B, dweights=C, renorm=0, scale=1.0, out=H, ldd=16, stream=None)
    a.update(change)
    assert _lib.load().sgemm_route_grad(*a.values()) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(type=3), dict(T=-1), dict(k=-1), dict(R=-1), dict(H=-1), dict(E=-1), dict(ldx=31), dict(X=0), dict(X=A + 1), dict(slots=0),
    dict(slots=B + 2), dict(offsets=0), dict(Y=0), dict(ldy=31), dict(Y=A + 64), dict(Y=B), dict(Y=D), dict(T=2 ** 30, k=2)], ids=str)
def test_spread_refuses(change):
    a = dict(type=1, T=8, k=2, R=16, H=32, X=A, ldx=32, slots=B, E=4, offsets=D, Y=C, ldy=32, stream=None)
    a.update(change)
    assert _lib.load().sgemm_spread(*a.values()) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(type=3), dict(T=-1), dict(R=-1), dict(ldy=31), dict(Y=0), dict(slots=0), dict(weights=D + 1), dict(out=0), dict(ldo=31),
    dict(out=A + 64), dict(out=B), dict(out=D)], ids=str)
def test_combine_refuses(change):
    a = dict(type=1, T=8, k=2, R=16, H=32, Y=A, ldy=32, slots=B, weights=D, out=C, ldo=32, stream=None)
    a.update(change)
    assert _lib.load().sgemm_combine(*a.values()) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(type=3), dict(T=-1), dict(ldd=31), dict(dout=0), dict(Y=0), dict(ldy=31), dict(slots=0), dict(weights=D + 1), dict(offsets=0),
    dict(lddy=31), dict(dY=A), dict(dY=B + 32), dict(dweights=C), dict(dweights=A), dict(E=-1), dict(dY=H)], ids=str)
def test_combine_grad_refuses(change):
    a = dict(type=1, T=8, k=2, R=16, H=32, dout=A, ldd=32, Y=B, ldy=32, slots=C, weights=D, E=4, offsets=F, dY=H + 4096, lddy=32,
             dweights=H, stream=None)
    a.update(change)
    assert _lib.load().sgemm_combine_grad(*a.values()) == _lib.ERR_INVALID_ARG


def test_entries_without_work_touch_no_device():
    lib = _lib.load()
    assert lib.sgemm_spread(1, 0, 2, 0, 32, 0, 32, 0, 4, D, 0, 32, None) == _lib.OK
    assert lib.sgemm_combine(1, 0, 2, 16, 32, A, 32, 0, 0, 0, 32, None) == _lib.OK
    assert lib.sgemm_combine_grad(1, 8, 2, 16, 32, A, 32, 0, 32, B, 0, 0, 0, 0, 32, 0, None) == _lib.OK
    assert lib.sgemm_route_grad(1, 0, 0, 16, 2, 0, 16, 0, 0, 0, 1.0, 0, 16, None) == _lib.OK


def test_binding_refuses_cpu_tensors():
    x, i = torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: g.sgemm_route(x, 2), lambda: g.sgemm_route_grad(x, i, torch.zeros(4, 2)), lambda: g.sgemm_spread(x, i, i[:, 0]),
                 lambda: g.sgemm_combine(x, i), lambda: g.sgemm_combine_grad(x, x, i, None, i[:, 0])):
        with pytest.raises(TypeError):
            call()


def test_header_states_which_entry_points_allocate():
    import os
    import re

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sgemm_routing.h")
    text = open(path).read()
    listed = [re.search(rf"\* +{tag}: ([\w ]+)", text).group(1).split() for tag in ("ROUTING-ALLOCATING", "ROUTING-NON-ALLOCATING")]
    declared = re.findall(r"^int (sgemm_\w+)\(", text, flags=re.M)
    assert sorted(listed[0] + listed[1]) == sorted(declared)


# ------------------------------------------------------------------ routing

HOW = [
    dict(),
    dict(renormalize=True, scale=2.5),
    dict(score="sigmoid"),
    dict(score="sigmoid", renormalize=True, scale=0.5),
]


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("how", HOW, ids=str)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 4), (2, 8, 8), (31, 33, 5), (32, 32, 32), (33, 128, 6), (65, 40, 3), (100, 257, 9),
                                   (70, 500, 17), (40, 1024, 32), (260, 60, 2)])
def test_route(T, E, k, how, bias, dtype):
    logits = randn(T, E, seed=T + E, dtype=dtype)
    b = 0.1 * randn(E, seed=3) if bias else None
    check_route(g.sgemm_route(logits, k, bias=b, **how), logits, k, bias=b, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (64, 8, 3, 6), (40, 5, 2, 9), (36, 4, 1, 4), (12, 6, 3, 6), (1024, 32, 5, 20),
                                            (30, 30, 7, 7), (96, 3, 2, 4), (256, 16, 1, 16), (64, 2, 2, 5)])
def test_route_by_groups(E, groups, top, k, best, bias, score):
    logits = randn(50, E, seed=E + groups, dtype=torch.bfloat16)
    b = 0.1 * randn(E, seed=4) if bias else None
    how = dict(score=score, bias=b, groups=groups, top_groups=top, group_best=best, renormalize=True)
    check_route(g.sgemm_route(logits, k, **how), logits, k, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("how", [dict(), dict(score="sigmoid", renormalize=True), dict(groups=4, top_groups=2, group_best=2)], ids=str)
@pytest.mark.parametrize("bias", [False, True])
def test_route_experts_out_of_service(how, bias):
    """-inf logits: some experts, all but a few, all; a -inf bias closes an expert for the choice."""
    T, E, k = 80, 32, 6
    logits = randn(T, E, seed=5)
    logits[:, 3] = -INF
    logits[10:20, 4:] = -INF       # three experts left
    logits[20:30] = -INF           # none
    logits[30] = -INF
    logits[30, 31] = -200.0        # one, of a score that is 0 in float32 as a sigmoid
    logits[31:33] = torch.finfo(torch.float32).min  # the lowest values: in service
    b = None
    if bias:
        b = 0.1 * randn(E, seed=6)
        b[7] = -INF
    r = g.sgemm_route(logits, k, bias=b, **how)
    check_route(r, logits, k, bias=b, **how)
    assert (r.experts[20:30] == -1).all() and (r.weights[20:30] == 0).all() and (r.slots[20:30] == -1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("how", [dict(), dict(score="sigmoid", renormalize=True), dict(groups=4, top_groups=2, group_best=2),
                                 dict(groups=4, top_groups=2, group_best=1)], ids=str)
@pytest.mark.parametrize("bias", [False, True])
def test_route_ties_go_to_the_lowest(how, bias):
    """Equal logits, of few values, and zeros of either sign."""
    T, E, k = 64, 48, 7
    gen = torch.Generator(device="cuda").manual_seed(7)
    logits = torch.randint(-1, 2, (T, E), generator=gen, device="cuda").float()
    logits[0] = 0
    logits[1] = torch.where(torch.arange(E, device="cuda") % 2 == 0, 0.0, -0.0)
    b = torch.zeros(E, device="cuda") if bias else None
    check_route(g.sgemm_route(logits, k, bias=b, **how), logits, k, bias=b, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_decides_near_values_exactly(score):
    """Biases that make choices differ in their 30th bit only: c_e = s_e + b_e with b_e = float32(1/2 - s_e), so that each c
    is 1/2 but for the bias's rounding (2^-26) and float32 could not tell them apart."""
    E, k = 64, 8
    l = randn(1, E, seed=8)
    b = (0.5 - scores64(l, score))[0].float()
    logits = l.expand(40, E).contiguous()
    check_route(g.sgemm_route(logits, k, score=score, bias=b), logits, k, score=score, bias=b)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_route_non_finite_logits_stay_in_their_token(bad, bias, score):
    T, E, k = 40, 64, 4
    logits = randn(T, E, seed=9)
    b = 0.1 * randn(E, seed=10) if bias else None
    want = g.sgemm_route(logits, k, score=score, bias=b, renormalize=True)
    broken = logits.clone()
    broken[17, 5] = bad
    r = g.sgemm_route(broken, k, score=score, bias=b, renormalize=True)
    keep = torch.arange(T, device="cuda") != 17
    assert torch.equal(r.experts[keep], want.experts[keep]) and torch.equal(r.weights[keep], want.weights[keep])
    assert ((r.experts >= 0) & (r.experts < E)).all() and len(set(r.experts[17].tolist())) == k
    if bad != bad or score == "softmax":
        assert r.weights[17].isnan().all()
    else:
        assert r.experts[17, 0] == 5 or bias
    offsets, slots = places64(r.experts.cpu(), E)
    assert torch.equal(r.offsets.cpu(), offsets) and torch.equal(r.slots.cpu(), slots)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [-90.0, -300.0, 60.0])
def test_renormalised_weights_of_scores_at_the_ends(shift):
    """Scores that float32 cannot hold (sigmoid(-300)) still have their ratios."""
    logits = randn(20, 16, seed=11) + shift
    for how in (dict(score="sigmoid", renormalize=True), dict(renormalize=True)):
        check_route(g.sgemm_route(logits, 3, **how), logits, 3, **how)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (0, 8), (3, 0), (1, 5)])
def test_route_strides_and_alignment(pad, shift, dtype):
    T, E, k = 75, 72, 4
    logits = randn(T, E, seed=12, dtype=dtype)
    b = 0.1 * randn(E, seed=13)
    r = g.sgemm_route(padded(logits, pad, shift), k, bias=b)
    check_route(r, logits, k, bias=b)
    d = randn(T, k, seed=14)
    out = padded(torch.zeros((T, E), dtype=dtype, device="cuda"), pad, shift)
    whole = out.untyped_storage()
    dl = g.sgemm_route_grad(padded(logits, pad, shift), r.experts, d, out)
    assert dl is out
    check_route_grad(dl, logits, r.experts, d)
    store = torch.empty(0, dtype=dtype, device="cuda").set_(whole, 0, (whole.nbytes() // out.element_size(),), (1,))
    assert int(store.isnan().sum()) == shift + T * pad, "padding was written"


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(5000, 16, 2), (20000, 8, 1), (11111, 300, 3)])
def test_route_many_tokens(T, E, k):
    """Several steps and many CTAs; the choice itself is checked by torch's sort, places by a stable sort."""
    logits = randn(T, E, seed=15)
    logits[T // 2: T // 2 + 700] = -INF
    r = g.sgemm_route(logits, k, renormalize=True)
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k].int()
    order[T // 2: T // 2 + 700] = -1
    assert torch.equal(r.experts, order)
    key = torch.where(order.flatten() < 0, E, order.flatten())
    at = torch.argsort(key, stable=True)
    slots = torch.empty_like(key)
    slots[at] = torch.arange(T * k, device="cuda", dtype=torch.int32)
    slots[key == E] = -1
    assert torch.equal(r.slots.flatten(), slots)
    offsets = torch.zeros(E + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0)
    assert torch.equal(r.offsets, offsets.int())
    again = g.sgemm_route(logits, k, renormalize=True)
    assert all(torch.equal(x, y) for x, y in zip(r, again))


@pytest.mark.gpu
def test_route_of_no_tokens():
    r = g.sgemm_route(torch.zeros((0, 8), device="cuda"), 2)
    assert r.experts.shape == (0, 2) and r.slots.shape == (0, 2) and r.offsets.tolist() == [0] * 9
    assert g.sgemm_route_grad(torch.zeros((0, 8), device="cuda"), r.experts, r.weights).shape == (0, 8)


# ------------------------------------------------------------------ gradient of the routing


def weights64(l, experts, score, renormalize, scale):
    there = experts >= 0
    if renormalize and score == "softmax":  # (of the chosen alone: the others' gradients are zeros, and not cancelled sums)
        x = torch.gather(l.double(), 1, experts.clamp(min=0).long())
        x = torch.where(there, x, torch.where(there.any(-1, keepdim=True), -INF, 0.0))
        return scale * torch.softmax(x, -1) * there
    closed = (l == -INF).all(-1, keepdim=True)
    s = scores64(torch.where(closed, 0.0, l.double()), score)
    w = torch.gather(s, 1, experts.clamp(min=0).long()) * there
    if renormalize:
        w = w / torch.where(there.any(-1, keepdim=True), w.sum(-1, keepdim=True), 1.0)
    return scale * w


def check_route_grad(dl, logits, experts, d, score="softmax", renormalize=False, scale=1.0):
    dtype = dl.dtype
    l = logits.double().clone().requires_grad_()
    there = experts >= 0
    d = torch.where(there, d.double(), 0.0)
    (weights64(l, experts, score, renormalize, scale) * d).sum().backward()
    exact = torch.where(l.isfinite(), torch.nan_to_num(l.grad), 0.0)
    s = scores64(torch.where((l == -INF).all(-1, keepdim=True), 0.0, l), score).detach()
    at = experts.clamp(min=0).long()
    sj = torch.gather(s, 1, at) * there
    if renormalize:  # (the chosen scores' shares)
        share = sj / torch.where(there.any(-1, keepdim=True), sj.sum(-1, keepdim=True), 1.0)
        s = torch.zeros_like(s).scatter_add(1, at, share)
        sj = share
    da = torch.zeros_like(s).scatter_add(1, at, d.abs())
    bound = scale * s * (da + (sj * d.abs()).sum(-1, keepdim=True))
    limit = 2.0 ** -18 * bound + U[dtype] * exact.abs() + TINY[dtype]
    assert ((dl.double() - exact).abs() <= limit * 1.001).all(), ((dl.double() - exact).abs() / limit).max()


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("how", HOW, ids=str)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 64, 4), (31, 33, 5), (100, 257, 9), (70, 500, 17), (40, 1024, 32), (9, 12, 12)])
def test_route_gradient(T, E, k, how, dtype):
    logits = randn(T, E, seed=20 + T, dtype=dtype)
    logits[T // 2, : E // 2] = -INF
    if T > 4:
        logits[3] = -INF
    r = g.sgemm_route(logits, k, **how)
    d = randn(T, k, seed=21)
    d[r.experts < 0] = NAN  # (of choices that are none: not read)
    check_route_grad(g.sgemm_route_grad(logits, r.experts, d, **how), logits, r.experts, d, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("how", HOW, ids=str)
def test_route_gradient_against_differences(how):
    """Central differences of L = sum(weights * R) in 64 bits, step h = 2^-10: the third derivative of a score is below 2, so
    the difference is off by h^2 sum |R| 2 scale / 3 at most, and the kernel by 2^-18 scale sum |R|."""
    T, E, k, h = 4, 12, 3, 2.0 ** -10
    logits = randn(T, E, seed=22)
    r = g.sgemm_route(logits, k, **how)
    R = randn(T, k, seed=23)
    dl = g.sgemm_route_grad(logits, r.experts, R, **how).double()
    score, renormalize, scale = how.get("score", "softmax"), how.get("renormalize", False), how.get("scale", 1.0)
    for e in range(E):
        step = torch.zeros((1, E), dtype=torch.float64, device="cuda")
        step[0, e] = h
        hi, lo = (weights64(logits.double() + s * step, r.experts, score, renormalize, scale) * R.double() for s in (1, -1))
        diff = (hi - lo).sum(-1) / (2 * h)
        limit = R.double().abs().sum(-1) * scale * (2 * h * h + 2.0 ** -17)
        assert ((dl[:, e] - diff).abs() <= limit).all()


# ------------------------------------------------------------------ rows

ROWS = [(1, 1, 1, 1), (1, 4, 8, 64), (3, 2, 4, 7), (40, 3, 8, 264), (65, 8, 16, 1027), (130, 1, 3, 136), (300, 6, 40, 520), (17, 11, 16, 2048),
        (700, 2, 5, 72), (9, 20, 64, 40)]


def routed(T, k, E, seed=30):
    logits = randn(T, E, seed=seed)
    if T > 8:
        logits[5:8] = -INF
    return g.sgemm_route(logits, k, renormalize=True)


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (2, 2), (1, 5)])
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_spread_and_combine(T, k, E, H, pad, shift, dtype):
    r = routed(T, k, E)
    X = randn(T, H, seed=31, dtype=dtype)
    R, used = T * k, int(r.offsets[-1])
    out = padded(torch.full((R, H), 7.0, dtype=dtype, device="cuda"), pad, shift)
    whole = out.untyped_storage()
    Y = g.sgemm_spread(padded(X, pad, shift), r.slots, r.offsets, out)
    want = torch.zeros((R, H), dtype=dtype, device="cuda")
    there = r.slots >= 0
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)
    want[r.slots[there].long()] = X[token[there]]
    assert torch.equal(Y, want) and (Y[used:] == 0).all()
    store = torch.empty(0, dtype=dtype, device="cuda").set_(whole, 0, (whole.nbytes() // out.element_size(),), (1,))
    assert int(store.isnan().sum()) == shift + R * pad, "padding was written"
    Y = randn(R, H, seed=32, dtype=dtype)
    Y[used:] = NAN  # (rows of no choice are not read)
    rows = torch.where(there[..., None], Y[r.slots.clamp(min=0).long()].double(), 0.0)
    for w in (None, r.weights):
        ww = torch.ones((T, k), dtype=torch.float64, device="cuda") if w is None else w.double()
        exact, bound = (rows * ww[..., None]).sum(1), (rows.abs() * ww.abs()[..., None]).sum(1)
        y = g.sgemm_combine(padded(Y, pad, shift), r.slots, w)
        limit = (k + 1) * 2.0 ** -24 * bound
        assert ((y.double() - exact).abs() <= limit + U[dtype] * (exact.abs() + limit) + TINY[dtype]).all()


@pytest.mark.gpu
@typed(TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 0), (2, 2)])
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_combine_gradient(T, k, E, H, pad, shift, dtype):
    r = routed(T, k, E)
    R, used = T * k, int(r.offsets[-1])
    Y, d = randn(R, H, seed=33, dtype=dtype), randn(T, H, seed=34, dtype=dtype)
    Y[used:] = NAN
    there = r.slots >= 0
    rows = torch.where(there[..., None], Y[r.slots.clamp(min=0).long()].double(), 0.0)
    for w in (r.weights, None):
        dY, dw = g.sgemm_combine_grad(padded(d, pad, shift), padded(Y, pad, shift), r.slots, w, r.offsets)
        ww = torch.ones((T, k), device="cuda") if w is None else w
        want = torch.zeros((R, H), dtype=torch.float64, device="cuda")
        want[r.slots[there].long()] = (ww.double()[..., None] * d.double()[:, None])[there]
        assert (dY[used:] == 0).all()
        limit = 2.0 ** -24 * want.abs()
        assert ((dY.double() - want).abs() <= limit + U[dtype] * (want.abs() + limit) + TINY[dtype]).all()
        exact, bound = (rows * d.double()[:, None]).sum(-1), (rows * d.double()[:, None]).abs().sum(-1)
        assert dw.dtype == torch.float32
        assert ((dw.double() - exact).abs() <= (H / 32 + 24) * 2.0 ** -24 * bound).all()
        only_rows, only_weights = (g.sgemm_combine_grad(d, Y, r.slots, w, r.offsets, needs=n) for n in ((True, False), (False, True)))
        assert only_rows[1] is None and torch.equal(only_rows[0], dY)
        assert only_weights[0] is None  # (the vectors' width, and so the order of a sum, goes by all operands' alignment)
        assert ((only_weights[1].double() - exact).abs() <= (H / 32 + 24) * 2.0 ** -24 * bound).all()


@pytest.mark.gpu
def test_rows_that_no_slot_names_and_slots_out_of_range():
    """A wider output than there are choices, slots past it or negative, rows below offsets[-1] that nobody names."""
    T, k, H, R = 6, 2, 40, 20
    X = randn(T, H, seed=35)
    slots = torch.tensor([[3, -1], [-5, 25], [2 ** 31 - 1, 19], [7, 8], [20, -2 ** 31], [0, 1]], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 4, 12], dtype=torch.int32, device="cuda")
    out = torch.full((R, H), 5.0, device="cuda")
    Y = g.sgemm_spread(X, slots, offsets, out)
    want = torch.full((R, H), 5.0, device="cuda")
    want[12:] = 0
    for s, t in ((3, 0), (7, 3), (8, 3), (0, 5), (1, 5)):
        want[s] = X[t]
    assert torch.equal(Y[:19], want[:19])  # (row 19 is named, and from offsets[-1] on)
    w = torch.rand((T, k), device="cuda")
    Y = randn(R, H, seed=36)
    y = g.sgemm_combine(Y, slots, w).double()
    want = torch.stack([w[0, 0] * Y[3], 0 * Y[0], w[2, 1] * Y[19], w[3, 0] * Y[7] + w[3, 1] * Y[8], 0 * Y[0], w[5, 0] * Y[0] + w[5, 1] * Y[1]]).double()
    assert ((y - want).abs() <= 2.0 ** -21 * want.abs().clamp(min=1)).all()
    dw = g.sgemm_combine_grad(X, Y, slots, w, offsets, needs=(False, True))[1]
    assert (dw != 0).tolist() == [[True, False], [False, False], [False, True], [True, True], [False, False], [True, True]]
    for bad in (-3, 2 ** 31 - 1):  # boundaries out of range: all rows, or none
        o = torch.tensor([0, bad], dtype=torch.int32, device="cuda")
        Y = g.sgemm_spread(X[:0], slots[:0], o, torch.full((R, H), 5.0, device="cuda"))
        assert (Y == (0 if bad < 0 else 5)).all()


@pytest.mark.gpu
@typed(TYPES)
def test_no_tokens_no_choices_no_columns(dtype):
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    empty = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    X = torch.zeros((0, 16), dtype=dtype, device="cuda")
    assert g.sgemm_spread(X, empty, o).shape == (0, 16)
    assert g.sgemm_combine(X, empty).shape == (0, 16)
    dY, dw = g.sgemm_combine_grad(X, X, empty, None, o)
    assert dY.shape == (0, 16) and dw.shape == (0, 2)
    none = torch.zeros((5, 0), dtype=torch.int32, device="cuda")
    Y = torch.ones((5, 16), dtype=dtype, device="cuda")
    assert (g.sgemm_combine(Y, none) == 0).all()
    slots = torch.arange(10, dtype=torch.int32, device="cuda").view(5, 2)
    narrow = torch.zeros((10, 0), dtype=dtype, device="cuda")
    assert g.sgemm_spread(narrow[:5], slots, o).shape == (10, 0)
    dY, dw = g.sgemm_combine_grad(narrow[:5], narrow, slots, None, o)
    assert dY.shape == (10, 0) and (dw == 0).all()


@pytest.mark.gpu
def test_binding_checks():
    x = randn(4, 8, seed=40)
    r = g.sgemm_route(x, 2)
    X = randn(4, 16, seed=41)
    for call in (lambda: g.sgemm_route(x, 0), lambda: g.sgemm_route(x, 9), lambda: g.sgemm_route(x, 2, score="max"),
                 lambda: g.sgemm_route(x, 2, groups=3), lambda: g.sgemm_route(x, 2, groups=4, top_groups=5),
                 lambda: g.sgemm_route(x, 2, group_best=3), lambda: g.sgemm_route(x, 2, bias=torch.zeros(7, device="cuda")),
                 lambda: g.sgemm_route(x.T, 2), lambda: g.sgemm_route_grad(x, r.experts[:3], r.weights[:3]),
                 lambda: g.sgemm_route_grad(x, r.experts, r.weights[:, :1]), lambda: g.sgemm_spread(X[:3], r.slots, r.offsets),
                 lambda: g.sgemm_spread(X, r.slots.T, r.offsets), lambda: g.sgemm_spread(X, r.slots, r.offsets[::2]),
                 lambda: g.sgemm_combine(X, r.slots, r.weights[:, :1]), lambda: g.sgemm_combine_grad(X, X[:, :8], r.slots, None, r.offsets)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.sgemm_route(x.double(), 2), lambda: g.sgemm_route(x, 2, bias=torch.zeros(8, device="cuda").half()),
                 lambda: g.sgemm_route_grad(x, r.experts.long(), r.weights), lambda: g.sgemm_spread(X, r.slots.long(), r.offsets),
                 lambda: g.sgemm_combine(X, r.slots, r.weights.half()), lambda: g.sgemm_combine_grad(X, X.half(), r.slots, None, r.offsets)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ together


def layer(logits, X, W, k, stream=None):
    r = g.sgemm_route(logits, k, score="sigmoid", renormalize=True, stream=stream)
    rows = g.sgemm_spread(X, r.slots, r.offsets, stream=stream)
    Y = g.sgemm_grouped(rows, W, r.offsets, stream=stream)
    return r, Y, g.sgemm_combine(Y, r.slots, r.weights, stream=stream)


def check_layer(y, logits, X, W, k):
    """A token's row through its experts in 64 bits.  The products' rows are rounded to bf16 once and their sum once more."""
    experts, weights = route64(logits, k, score="sigmoid", renormalize=True)
    exact, bound = torch.zeros_like(y, dtype=torch.float64), torch.zeros_like(y, dtype=torch.float64)
    for t in range(X.shape[0]):
        for j in range(k):
            e = int(experts[t, j])
            if e >= 0:
                exact[t] += weights[t, j].item() * (X[t].double() @ W[e].double())
                bound[t] += weights[t, j].item() * (X[t].double().abs() @ W[e].double().abs())
    u = U[torch.bfloat16]
    assert ((y.double() - exact).abs() <= 1.1e-4 * bound + 2.1 * u * bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 50])
def test_a_layer(T):
    E, K, N, k = 8, 72, 136, 2
    logits, X, W = randn(T, E, seed=50), randn(T, K, seed=51, dtype=torch.bfloat16), randn(E, K, N, seed=52, dtype=torch.bfloat16)
    check_layer(layer(logits, X, W, k)[2], logits, X, W, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = layer(logits, X, W, k, stream=side)[2]
    side.synchronize()
    check_layer(y, logits, X, W, k)
    assert g.check_status() == 0


@pytest.mark.gpu
def test_two_recorded_layers_on_two_streams():
    """Graphs replayed at the same time, whose calls take scratch of their own."""
    T, E, K, N, k = 600, 16, 64, 128, 3
    W = randn(E, K, N, seed=53, dtype=torch.bfloat16)
    logits = [torch.zeros((T, E), device="cuda") for _ in range(2)]
    X = [torch.zeros((T, K), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    layer(logits[0], X[0], W, k)
    graphs, out = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r, Y, y = layer(logits[i], X[i], W, k)
            d = g.sgemm_combine_grad(y, Y, r.slots, r.weights, r.offsets)
            dl = g.sgemm_route_grad(logits[i], r.experts, d[1], score="sigmoid", renormalize=True)
        graphs.append(graph)
        out.append((*r, Y, y, *d, dl))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for seed in range(3):
        for i in range(2):
            logits[i].copy_(randn(T, E, seed=60 + 2 * seed + i))
            X[i].copy_(randn(T, K, seed=70 + 2 * seed + i))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            r, Y, y = layer(logits[i], X[i], W, k)
            d = g.sgemm_combine_grad(y, Y, r.slots, r.weights, r.offsets)
            dl = g.sgemm_route_grad(logits[i], r.experts, d[1], score="sigmoid", renormalize=True)
            assert all(torch.equal(a, b) for a, b in zip((*r, Y, y, *d, dl), out[i]))
    assert g.check_status() == 0


@pytest.mark.gpu
def test_gradients_of_a_layer_against_differences():
    """Spread, combine and their gradients are linear: with integers of a few bits every product and sum is exact, and a
    central difference with step 1 is the gradient."""
    T, E, H, k = 12, 4, 24, 2
    r = routed(T, k, E, seed=54)
    gen = torch.Generator(device="cuda").manual_seed(55)
    ints = lambda *shape: torch.randint(-3, 4, shape, generator=gen, device="cuda").float()  # noqa: E731
    X, R, w = ints(T, H), ints(T * k, H), ints(T, k)
    dX = g.sgemm_combine(R, r.slots)
    loss = lambda x: (g.sgemm_spread(x, r.slots, r.offsets) * R).sum().item()  # noqa: E731
    for t, h in ((0, 0), (6, 3), (11, 23)):
        hi, lo = X.clone(), X.clone()
        hi[t, h] += 1
        lo[t, h] -= 1
        assert (loss(hi) - loss(lo)) / 2 == dX[t, h].item()
    Y, d = ints(T * k, H), ints(T, H)
    dY, dw = g.sgemm_combine_grad(d, Y, r.slots, w, r.offsets)
    loss = lambda y, v: (g.sgemm_combine(y, r.slots, v) * d).sum().item()  # noqa: E731
    for s, h in ((0, 0), (5, 7), (int(r.offsets[-1]) - 1, 23), (T * k - 1, 2)):
        hi, lo = Y.clone(), Y.clone()
        hi[s, h] += 1
        lo[s, h] -= 1
        assert (loss(hi, w) - loss(lo, w)) / 2 == dY[s, h].item()
    for t, j in ((0, 0), (6, 1), (11, 1)):
        hi, lo = w.clone(), w.clone()
        hi[t, j] += 1
        lo[t, j] -= 1
        assert (loss(Y, hi) - loss(Y, lo)) / 2 == dw[t, j].item()


@pytest.mark.gpu
@typed([torch.bfloat16])
def test_rows_past_2_31_elements(dtype):
    """Row numbers whose offsets do not fit 32 bits."""
    T, k, H = 3, 1, 2 ** 16
    R = 2 ** 15 + 3
    X = randn(T, H, seed=56, dtype=dtype)
    Y = torch.empty((R, H), dtype=dtype, device="cuda")
    slots = torch.tensor([[R - 1], [R - 2], [0]], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    g.sgemm_spread(X, slots, offsets, Y)
    assert torch.equal(Y[R - 1], X[0]) and torch.equal(Y[R - 2], X[1]) and torch.equal(Y[0], X[2])
    assert torch.equal(g.sgemm_combine(Y, slots), X)


