"""Measured cases of a layer of experts around its products: routing, the rows' way to their experts and back, and the
orthogonalised update of the experts' weights.

Four operators, each in a plain form of elementary torch operations and through the library's entry points:

* ``route``         a router's logits to every token's experts, their weights, and the rows' places by expert;
  ``route gradient`` its backward pass: the gradient of the logits from that of the weights;
* ``spread``        every token's row to the places of its choices, sorted by expert (its backward pass is ``combine``);
* ``combine``       the weighted sum of each token's rows, back in the tokens' order;
  ``combine gradient`` its backward pass: the gradient of the rows and of the weights;
* ``orthogonalize`` a weight update (or one for each expert) made orthogonal by Newton-Schulz products.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
# The quintic of the orthogonalisation, x -> a x + b x^3 + c x^5 on the singular values, and the number of steps.
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ------------------------------------------------------------------ cases


def listed():
    return [
        # One token of an interactive answer: latency is all that counts.
        {"name": "route one token bf16", "op": "route", "type": "bf16", "T": 1, "E": 64, "k": 4, "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "best": 1, "renorm": True, "scale": 1.0, "padded": 0, "closed": 0},
        # A long prompt over many small experts, balanced by a bias and limited to the best groups; a padded tail.
        {"name": "route prompt groups bf16", "op": "route", "type": "bf16", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "best": 2, "renorm": True, "scale": 2.5, "padded": 100, "closed": 0},
        # Odd sizes, a float32 router, some experts out of service, scores as they are.
        {"name": "route odd f32", "op": "route", "type": "f32", "T": 2047, "E": 40, "k": 3, "score": "softmax", "bias": True, "groups": 1,
         "top_groups": 1, "best": 1, "renorm": False, "scale": 1.0, "padded": 5, "closed": 3},
        # The router's part of a training step: a dense gradient (scores as they are) in float32 ...
        {"name": "route gradient step f32", "op": "route gradient", "type": "f32", "T": 8192, "E": 64, "k": 4, "score": "softmax",
         "renorm": False, "scale": 1.0, "padded": 0, "closed": 0},
        # ... and a sparse one for many experts.
        {"name": "route gradient many bf16", "op": "route gradient", "type": "bf16", "T": 16384, "E": 256, "k": 8, "score": "sigmoid",
         "renorm": True, "scale": 2.5, "padded": 100, "closed": 0},
        # A decoding batch on its way to its experts.
        {"name": "spread decode bf16", "op": "spread", "type": "bf16", "T": 64, "H": 4096, "E": 32, "k": 4, "padded": 3, "pad": 0},
        # A training step's rows.
        {"name": "spread step bf16", "op": "spread", "type": "bf16", "T": 8192, "H": 4096, "E": 64, "k": 4, "padded": 0, "pad": 0},
        # Row widths off the 16-byte grid, half precision.
        {"name": "combine odd f16", "op": "combine", "type": "f16", "T": 1023, "H": 1027, "E": 16, "k": 2, "padded": 9, "pad": 3},
        # The backward pass of a training step's combination.
        {"name": "combine gradient step bf16", "op": "combine gradient", "type": "bf16", "T": 8192, "H": 2048, "E": 64, "k": 8, "padded": 0, "pad": 0},
        # One small matrix at full precision: latency.
        {"name": "orthogonalize small f32", "op": "orthogonalize", "type": "f32", "E": 1, "M": 128, "N": 96, "rank": 4, "pad": 0},
        # Odd sizes, taller than wide, at full precision.
        {"name": "orthogonalize odd f32", "op": "orthogonalize", "type": "f32", "E": 2, "M": 1025, "N": 1023, "rank": 16, "pad": 1},
        # The weight gradients of a layer's experts in a training step.
        {"name": "orthogonalize experts bf16", "op": "orthogonalize", "type": "bf16", "E": 8, "M": 2048, "N": 4096, "rank": 64, "pad": 0},
    ]


def _spread_size(rng, lo, hi):
    """A size between lo and hi, even in its logarithm: a multiple of 128, of 8, or any."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice((1, 8, 128))
    if step > 1 and v >= step:
        v -= v % step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("route", "route", "route gradient", "spread", "combine", "combine gradient", "orthogonalize", "orthogonalize"))
    t = rng.choice(("bf16", "f16", "f32"))
    if op == "orthogonalize":
        M, N = _spread_size(rng, 32, 4096), _spread_size(rng, 32, 4096)
        short, long = min(M, N), max(M, N)
        # (2^37 a step, 0.3 of the largest listed case's: at full precision each costs more)
        most = 2 ** 37 // (3 * short * short * long + short ** 3)
        return {"op": op, "type": t, "E": max(1, min(most, rng.choice((1, 1, 2, 4, 8)))), "M": M, "N": N, "rank": rng.choice((0, 4, 16, 64)),
                "pad": rng.choice((0, 0, 1, 8))}
    T = _spread_size(rng, 1, 16384)
    E = rng.choice((4, 8, 16, 40, 60, 64, 128, 160, 256, 512))
    k = rng.randint(1, min(8, E // 2))
    case = {"op": op, "type": t, "T": T, "E": E, "k": k, "padded": rng.choice((0, 0, T // 10))}
    if op in ("route", "route gradient"):
        case |= {"score": rng.choice(("softmax", "sigmoid")), "renorm": rng.choice((True, False)), "scale": rng.choice((1.0, 2.5)),
                 "closed": rng.choice((0, 0, E // 8))}
        if op == "route gradient":
            case["renorm"] &= k > 1  # (a single renormalised weight is a constant)
        else:
            # (groups of at least 4 experts, so that half of the groups hold k that are in service)
            groups = rng.choice((1, 1, 4, 8))
            groups = groups if E % groups == 0 and E >= 4 * groups and E // 4 >= k else 1
            case |= {"bias": rng.choice((True, False)), "groups": groups, "top_groups": max(1, groups // 2), "best": rng.choice((1, 2))}
        return case
    H = _spread_size(rng, 64, min(8192, max(64, (1 << 27) // (T * k))))
    return case | {"H": H, "pad": rng.choice((0, 0, 8, 3))}


def work(case):
    s = BYTES[case["type"]]
    if case["op"] == "orthogonalize":
        m, n = min(case["M"], case["N"]), max(case["M"], case["N"])
        # (X X^T and A A are symmetric: each element once)
        return {"bytes": 2 * s * case["E"] * m * n, "flops": STEPS * case["E"] * (3 * m * m * n + m ** 3)}
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        return {"bytes": s * T * E + 12 * T * k + 4 * (E + 1), "flops": 0}
    if case["op"] == "route gradient":
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": s * T * E + (s * T * E if dense else s * T * k) + 8 * T * k, "flops": 0}
    R, H = T * k, case["H"]
    if case["op"] == "spread":
        return {"bytes": s * (T + R) * H + 4 * R, "flops": 0}
    if case["op"] == "combine":
        return {"bytes": s * (T + R) * H + 8 * R, "flops": 2 * R * H}
    return {"bytes": s * (T + 2 * R) * H + 12 * R, "flops": 3 * R * H}


# ------------------------------------------------------------------ inputs


def _rows(rows, case, g):
    """Rows in a buffer `pad` columns wider; a few channels far larger than the rest, as activations have them."""
    x = torch.randn((rows, case["H"] + case["pad"]), generator=g, device="cuda", dtype=torch.float32)
    x[:, 5::97] *= 8
    return x.to(DTYPES[case["type"]])[:, : case["H"]]


def _logits(case, g):
    """A router's logits: some experts wanted more than others; padding tokens and experts out of service at -inf."""
    T, E = case["T"], case["E"]
    x = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    x = x.to(DTYPES[case["type"]])
    if case["closed"]:
        x[:, torch.randperm(E, generator=g, device="cuda")[: case["closed"]]] = -math.inf
    if case["padded"]:
        x[T - case["padded"]:] = -math.inf
    return x


def _places(experts, E):
    """Boundaries of the experts' rows, and each choice's row when all choices are sorted by expert (-1: no expert)."""
    flat = experts.flatten().long()
    key = torch.where(flat < 0, E, flat)
    order = torch.argsort(key, stable=True)
    slots = torch.empty_like(order)
    slots[order] = torch.arange(flat.numel(), device=flat.device)
    count = torch.zeros(E + 1, dtype=torch.long, device=flat.device).index_add(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.cumsum(count[:E], 0)
    return offsets, torch.where(flat < 0, -1, slots).to(torch.int32).view(experts.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, t = case["op"], DTYPES[case["type"]]
    state = {"op": op, "case": case}
    if op == "orthogonalize":
        # A gradient as training gives it: a few strong directions over a floor of noise, small in absolute terms.
        E, M, N, r = case["E"], case["M"], case["N"], case["rank"]
        G = torch.randn((E, M, N + case["pad"]), generator=g, device="cuda")
        if r:
            u, v = torch.randn((E, M, r), generator=g, device="cuda"), torch.randn((E, r, N + case["pad"]), generator=g, device="cuda")
            G = 0.2 * G + u @ v / math.sqrt(r)
        state["G"] = (G * 1e-3).to(t)[..., :N]
        return state
    T, E, k = case["T"], case["E"], case["k"]
    if op in ("route", "route gradient"):
        state["logits"] = _logits(case, g)
        if op == "route":
            state["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        else:
            l = state["logits"].double()
            order = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, :k]
            state["experts"] = torch.where(torch.gather(l, 1, order) == -math.inf, -1, order).to(torch.int32)
            state["dweights"] = torch.randn((T, k), generator=g, device="cuda")
        return state
    # Choices as a router makes them: k experts that differ, some wanted more than others; padding tokens have none.
    order = torch.sort(torch.rand((T, E), generator=g, device="cuda") + torch.rand((1, E), generator=g, device="cuda"), -1).indices[:, :k]
    experts = order.to(torch.int32)
    experts[T - case["padded"]:] = -1
    state["offsets"], state["slots"] = _places(experts, E)
    if op == "spread":
        state["X"] = _rows(T, case, g)
        return state
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    state["weights"] = w / w.sum(-1, keepdim=True) * (experts >= 0)
    state["Y"] = _rows(T * k, case, g)
    if op == "combine gradient":
        state["dout"] = torch.randn((T, case["H"]), generator=g, device="cuda").to(t)
    return state


# ------------------------------------------------------------------ plain forms


def _scores(x, score):
    """Softmax (rows without an expert in service: zeros) or sigmoid, in x's precision."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0, m))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-300 if x.dtype == torch.float64 else 1e-38)


def _route(case, logits, bias):
    T, E, k = case["T"], case["E"], case["k"]
    # (in 64 bits: which of two near scores is larger decides whole numbers)
    l = logits.double()
    s = _scores(l, case["score"])
    c = s if bias is None else s + bias.double()
    c = torch.where(l == -math.inf, -math.inf, c)
    if case["groups"] > 1:
        by_group = torch.sort(c.view(T, case["groups"], -1), dim=-1, descending=True).values[..., : case["best"]]
        there = by_group[..., 0] > -math.inf
        group = torch.where(there, torch.where(by_group == -math.inf, 0, by_group).sum(-1), -math.inf)
        kept = torch.sort(group, dim=-1, descending=True, stable=True).indices[:, : case["top_groups"]]
        of = torch.arange(E, device=c.device) // (E // case["groups"])
        c = torch.where((kept[:, :, None] == of).any(1), c, -math.inf)
    best = torch.sort(c, dim=-1, descending=True, stable=True)
    there = best.values[:, :k] > -math.inf
    experts = best.indices[:, :k]
    w = torch.where(there, torch.gather(s, 1, experts).float(), 0)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-38)
    experts = torch.where(there, experts, -1).to(torch.int32)
    offsets, slots = _places(experts, E)
    return {"experts": experts, "weights": (w * case["scale"]).float(), "offsets": offsets, "slots": slots}


def _route_gradient(case, logits, experts, dweights):
    s = _scores(logits.float(), case["score"])
    there = experts >= 0
    at = experts.clamp(min=0).long()
    sj = torch.gather(s, 1, at) * there
    ds = case["scale"] * dweights * there
    if case["renorm"]:
        total = sj.sum(-1, keepdim=True).clamp(min=1e-38)
        ds = (ds - (ds * sj).sum(-1, keepdim=True) / total) / total * there
    if case["score"] == "sigmoid":
        return torch.zeros_like(s).scatter_add(1, at, ds * sj * (1 - sj)).to(logits.dtype)
    inner = (ds * sj).sum(-1, keepdim=True)
    return (s * (torch.zeros_like(s).scatter_add(1, at, ds) - inner)).to(logits.dtype)


def _orthogonalize(G):
    a, b, c = QUINTIC
    X = G.float()
    if G.shape[-2] > G.shape[-1]:
        X = X.mT
    X = X / (X.double().square().sum((-2, -1), keepdim=True).sqrt() + EPS).float()
    for _ in range(STEPS):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.mT if G.shape[-2] > G.shape[-1] else X).to(G.dtype).contiguous()


def _plain(state):
    op, case = state["op"], state["case"]
    if op == "route":
        return _route(case, state["logits"], state["bias"])
    if op == "route gradient":
        return _route_gradient(case, state["logits"], state["experts"], state["dweights"])
    if op == "orthogonalize":
        return _orthogonalize(state["G"])
    slots, t = state["slots"], DTYPES[case["type"]]
    there, at = slots >= 0, slots.clamp(min=0).long()
    if op == "spread":
        Y = torch.zeros((slots.numel(), case["H"]), dtype=t, device=slots.device)
        row = torch.arange(case["T"], device=slots.device)[:, None].expand_as(slots)
        Y[slots[there].long()] = state["X"][row[there]]
        return Y
    rows = state["Y"][at].float() * there[..., None]
    if op == "combine":
        return (rows * state["weights"][..., None]).sum(1).to(t)
    dout = state["dout"].float()
    dY = torch.zeros((slots.numel(), case["H"]), dtype=t, device=slots.device)
    dY[slots[there].long()] = (state["weights"][..., None] * dout[:, None])[there].to(t)
    return {"dY": dY, "dweights": (rows * dout[:, None]).sum(-1)}


# ------------------------------------------------------------------ the library's entry points


def _library(state):
    import dense_fp32_gemm_f32_gb300 as g

    op, case = state["op"], state["case"]
    if op == "route":
        r = g.sgemm_route(state["logits"], case["k"], score=case["score"], bias=state["bias"], groups=case["groups"],
                          top_groups=case["top_groups"], group_best=case["best"], renormalize=case["renorm"], scale=case["scale"])
        return {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "slots": r.slots}
    if op == "route gradient":
        return g.sgemm_route_grad(state["logits"], state["experts"], state["dweights"], score=case["score"], renormalize=case["renorm"],
                                  scale=case["scale"])
    if op == "spread":
        return g.sgemm_spread(state["X"], state["slots"], state["offsets"])
    if op == "combine":
        return g.sgemm_combine(state["Y"], state["slots"], state["weights"])
    if op == "combine gradient":
        dY, dweights = g.sgemm_combine_grad(state["dout"], state["Y"], state["slots"], state["weights"], state["offsets"])
        return {"dY": dY, "dweights": dweights}
    return g.sgemm_orthogonalize(state["G"], steps=STEPS, coefficients=QUINTIC, eps=EPS)


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _exact_choice(case, state):
    """Each token's experts, best first, and its scores, by looking for the largest again and again."""
    l = state["logits"].double()
    T, E = l.shape
    open_ = l > -math.inf
    if case["score"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.nan_to_num(torch.softmax(l, -1), nan=0.0)
    c = (s + state["bias"].double()) if state["bias"] is not None else s.clone()
    c[~open_] = -math.inf
    if case["groups"] > 1:
        size = E // case["groups"]
        score = torch.full((T, case["groups"]), -math.inf, dtype=torch.float64, device=l.device)
        for q in range(case["groups"]):
            part = c[:, q * size: (q + 1) * size].clone()
            for i in range(case["best"]):
                top = part.max(1)
                gain = torch.where(top.values > -math.inf, top.values, 0.0 if i else -math.inf)
                score[:, q] = gain if i == 0 else score[:, q] + gain
                part.scatter_(1, top.indices[:, None], -math.inf)
        left = torch.ones((T, case["groups"]), dtype=torch.bool, device=l.device)
        index = torch.arange(case["groups"], device=l.device)
        for _ in range(case["top_groups"]):
            best = torch.where(left, score, -math.inf).max(1, keepdim=True).values
            first = torch.where(left & (score == best), index, case["groups"]).min(1, keepdim=True).values
            left &= index != first
        c = torch.where(left.repeat_interleave(size, 1), -math.inf, c)
    index, experts = torch.arange(E, device=l.device), []
    for _ in range(case["k"]):
        best = c.max(1, keepdim=True).values
        first = torch.where(c == best, index, E).min(1, keepdim=True).values
        experts.append(torch.where(best > -math.inf, first, -1))
        c = torch.where(index == first, -math.inf, c)
    return torch.cat(experts, 1), s


def _exact_route(case, state):
    T, E, k = case["T"], case["E"], case["k"]
    experts, s = _exact_choice(case, state)
    w = torch.gather(s, 1, experts.clamp(min=0)) * (experts >= 0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0)
    flat = experts.flatten()
    offsets = torch.tensor([int((flat < e).sum() - (flat < 0).sum()) for e in range(E + 1)], device=flat.device)
    slots = torch.full_like(flat, -1)
    for e in range(E):
        mine = flat == e
        slots[mine] = offsets[e] + torch.arange(int(mine.sum()), device=flat.device)
    return {"experts": experts.int(), "weights": w * case["scale"], "offsets": offsets.int(), "slots": slots.view(T, k).int()}


def _exact_route_gradient(case, state):
    """By automatic differentiation of the weights' definition."""
    l = state["logits"].double()
    padded = (l == -math.inf).all(1, keepdim=True)
    x = torch.where(padded, 0.0, l).requires_grad_()
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, -1)
    there = state["experts"] >= 0
    w = torch.gather(s, 1, state["experts"].clamp(min=0).long()) * there
    if case["renorm"]:
        w = w / torch.where(there.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
    (d,) = torch.autograd.grad((w * case["scale"] * state["dweights"].double() * there).sum(), x)
    return torch.where(padded, 0.0, d)


def _exact_orthogonal(G):
    """The quintic on the singular values, with the orthogonal factors left where they are."""
    a, b, c = QUINTIC
    out = []
    for x in G.double():
        x = x / (torch.linalg.vector_norm(x) + EPS)
        tall = x.shape[0] > x.shape[1]
        for _ in range(STEPS):
            gram = x.T @ x if tall else x @ x.T
            poly = b * gram + torch.linalg.matrix_power(gram, 2) * c
            poly.diagonal().add_(a)
            x = x @ poly if tall else poly @ x
        out.append(x)
    return torch.stack(out)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, state)
    if op == "route gradient":
        return _exact_route_gradient(case, state)
    if op == "orthogonalize":
        return _exact_orthogonal(state["G"])
    slots, T, H = state["slots"], case["T"], case["H"]
    if op == "spread":
        Y = torch.zeros((slots.numel(), H), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = torch.nonzero(slots[:, j] >= 0)[:, 0]
            Y[slots[t, j].long()] = state["X"][t].double()
        return Y
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    dY = torch.zeros((slots.numel(), H), dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, case["k"]), dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        t = torch.nonzero(slots[:, j] >= 0)[:, 0]
        at = slots[t, j].long()
        w, rows = state["weights"][t, j].double()[:, None], state["Y"][at].double()
        if op == "combine":
            out[t] += w * rows
        else:
            dY[at] = w * state["dout"][t].double()
            dw[t, j] = torch.einsum("th,th->t", state["dout"][t].double(), rows)
    return out if op == "combine" else {"dY": dY, "dweights": dw}
