"""Measured cases of the grouped (ragged, by expert) products and of the 4-bit microscaled (MXFP4) operators.

Five operators, each in a plain form of elementary torch operations in 32 bits and through the library's entry points:

* ``forward``   rows sorted by expert times their expert's weights;
* ``gradient``  its backward pass: the gradient of the rows and of every expert's weights;
* ``quantize``  MXFP4 quantisation, and the values that the codes stand for read back;
* ``linear``    rows quantised and multiplied by one MXFP4 weight matrix;
* ``experts``   rows sorted by expert, quantised and multiplied by their expert's MXFP4 weights.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
# Magnitudes of the 4-bit values (2 exponent bits, 1 mantissa bit), by code.
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases


def listed():
    return [
        # One token of an interactive answer: a single row finds one of 8 experts; latency is all that counts.
        {"name": "forward one row bf16", "op": "forward", "type": "bf16", "T": 1, "E": 8, "K": 1024, "N": 2048, "skew": 0.5, "pad": 0},
        # A decoding batch: two rows an expert on average, some with none; the weights' bytes count.
        {"name": "forward decode bf16", "op": "forward", "type": "bf16", "T": 64, "E": 32, "K": 2048, "N": 4096, "skew": 0.5, "pad": 0},
        # A long prompt or a training step's rows: the product's rate counts.
        {"name": "forward prompt bf16", "op": "forward", "type": "bf16", "T": 16384, "E": 16, "K": 4096, "N": 4096, "skew": 0.5, "pad": 0},
        # Odd sizes in every direction, in the library's own type, rows in a wider buffer.
        {"name": "forward odd f32", "op": "forward", "type": "f32", "T": 2047, "E": 8, "K": 1025, "N": 1023, "skew": 1.0, "pad": 3},
        # Fine-tuning on a short batch: few rows an expert, half precision, row widths off the 16-byte grid.
        {"name": "gradient short f16", "op": "gradient", "type": "f16", "T": 1023, "E": 16, "K": 1027, "N": 1020, "skew": 1.0, "pad": 0},
        # The backward pass of a training step.
        {"name": "gradient step bf16", "op": "gradient", "type": "bf16", "T": 8192, "E": 8, "K": 4096, "N": 2048, "skew": 0.5, "pad": 0},
        # The same in float32, for a master copy trained at full precision.
        {"name": "gradient step f32", "op": "gradient", "type": "f32", "T": 2048, "E": 4, "K": 1024, "N": 2048, "skew": 0.5, "pad": 0},
        # A decoding batch's activations.
        {"name": "quantize rows bf16", "op": "quantize", "type": "bf16", "T": 16, "K": 4096, "pad": 0},
        # A weight matrix converted from its float32 master copy.
        {"name": "quantize weights f32", "op": "quantize", "type": "f32", "T": 8192, "K": 8192, "pad": 0},
        # One token through one 4-bit projection: the weights' bytes count.
        {"name": "linear one row bf16", "op": "linear", "type": "bf16", "T": 1, "K": 8192, "N": 8192, "pad": 0},
        # A decoding batch through 4-bit experts.
        {"name": "experts decode bf16", "op": "experts", "type": "bf16", "T": 128, "E": 32, "K": 4096, "N": 2048, "skew": 0.5, "pad": 0},
        # A prompt through 4-bit experts: the product's rate counts.
        {"name": "experts prompt bf16", "op": "experts", "type": "bf16", "T": 16384, "E": 8, "K": 4096, "N": 8192, "skew": 0.5, "pad": 0},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even in its logarithm: a multiple of 128, of 8, or any."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice((1, 8, 128))
    if step > 1 and v >= step:
        v -= v % step
    if v == 3072:  # (no size of this repository's workloads)
        v += step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("forward", "forward", "gradient", "gradient", "quantize", "linear", "experts"))
    t = rng.choice(("bf16", "f16", "f32"))
    rows = 2048 if t == "f32" and op in ("forward", "gradient") else 8192
    case = {"op": op, "type": t, "T": _spread(rng, 1, rows), "K": _spread(rng, 64, 8192), "pad": rng.choice((0, 0, 8, 3))}
    if op in ("forward", "gradient", "experts"):
        case["E"] = rng.choice((1, 3, 8, 16, 40, 64))
        case["skew"] = rng.choice((0.0, 0.5, 1.0))
    if op != "quantize":
        # (at most 2^28 weights, what the largest listed cases hold; fewer where they take more bytes)
        held = {"gradient": 2, "forward": 1}.get(op, 0) * BYTES[t] // 2 or 1
        most = min(8192, (1 << 28) // (held * case["K"] * case.get("E", 1)))
        case["N"] = _spread(rng, 64, max(64, most))
    return case


def _shares(case):
    """The router's share of rows by expert, most wanted first."""
    p = [1.0 / (1 + e) ** case["skew"] for e in range(case["E"])]
    total = sum(p)
    return [v / total for v in p]


def work(case):
    T, K, s = case["T"], case["K"], BYTES[case["type"]]
    if case["op"] == "quantize":
        return {"bytes": 2 * s * T * K, "flops": 0}
    N = case["N"]
    if case["op"] == "linear":
        return {"bytes": s * T * (K + N) + N * K * 17 / 32, "flops": 2 * T * K * N}
    touched = sum(1 - (1 - p) ** T for p in _shares(case))
    if case["op"] == "forward":
        return {"bytes": s * (T * (K + N) + touched * K * N), "flops": 2 * T * K * N}
    if case["op"] == "gradient":  # rows and their gradient, weights of the experts met, all of the weights' gradient
        return {"bytes": s * (T * (2 * K + N) + (touched + case["E"]) * K * N), "flops": 4 * T * K * N}
    return {"bytes": s * T * (K + N) + touched * N * K * 17 / 32, "flops": 2 * T * K * N}


# ------------------------------------------------------------------ inputs


def _rows(case, width, g):
    """T rows in a buffer `pad` columns wider; a few channels far larger than the rest, as activations have them."""
    x = torch.randn((case["T"], width + case["pad"]), generator=g, device="cuda", dtype=torch.float32)
    x[:, 5::97] *= 8
    return x.to(DTYPES[case["type"]])[:, : width]


def _offsets(case, seed):
    """Boundaries of the experts' rows (E + 1), and the most rows that one of them has."""
    c = torch.Generator().manual_seed(seed)
    p = torch.tensor(_shares(case), dtype=torch.float64)[torch.randperm(case["E"], generator=c)]
    e = torch.multinomial(p, case["T"], replacement=True, generator=c)
    n = torch.bincount(e, minlength=case["E"])
    o = torch.zeros(case["E"] + 1, dtype=torch.int32)
    o[1:] = torch.cumsum(n, 0)
    return o.cuda(), int(n.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, K, t = case["T"], case["K"], DTYPES[case["type"]]
    state = {"op": case["op"], "type": t, "X": _rows(case, K, g)}
    if case["op"] in ("forward", "gradient", "experts"):
        state["offsets"], state["most"] = _offsets(case, seed)
    if case["op"] in ("forward", "gradient"):
        w = torch.randn((case["E"], K, case["N"]), generator=g, device="cuda", dtype=torch.float32)
        state["W"] = (w / math.sqrt(K)).to(t)
    if case["op"] == "gradient":
        state["dY"] = torch.randn((T, case["N"]), generator=g, device="cuda", dtype=torch.float32).to(t)
    if case["op"] in ("linear", "experts"):
        # MXFP4 weights, as a checkpoint holds them: two codes a byte (the even column in the low bits), and a byte
        # 127 + exponent for each 32 columns, laid out in blocks of 128 rows x 4 scales (see _scales_by_row).
        lead = (case["E"],) if case["op"] == "experts" else ()
        kb, N = (K + 31) // 32, case["N"]
        state["codes"] = torch.randint(0, 256, lead + (N, 16 * kb), generator=g, device="cuda", dtype=torch.uint8)
        if K % 32:  # columns past K hold zeros
            state["codes"][..., (K + 1) // 2:] = 0
            if K % 2:
                state["codes"][..., K // 2] &= 15
        nb, kq = (N + 127) // 128, (kb + 3) // 4
        state["scales"] = torch.randint(116, 122, lead + (nb, kq, 32, 4, 4), generator=g, device="cuda", dtype=torch.uint8)
    return state


# ------------------------------------------------------------------ plain forms


def _by_expert(x, offsets, most):
    """The experts' rows as (E, most, columns), zeros after each expert's last; the product of all experts is then one batched product."""
    at = offsets[:-1, None] + torch.arange(most, device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)].float() * (at < offsets[1:, None])[..., None]


def _by_row(y, offsets, T):
    """Rows of (E, most, columns) back in their order."""
    t = torch.arange(T, device=y.device)
    e = (t[:, None] >= offsets[None, 1:]).sum(1)
    return y[e, t - offsets[e]]


def _magnitudes(code):
    """The magnitude of each 3-bit code: 0, 1/2, 1, 3/2, 2, 3, 4, 6 (2 exponent bits, 1 mantissa bit)."""
    return torch.where(code < 2, code * 0.5, (2 + (code & 1)) * (1 << (code >> 1)) * 0.25)


def _rounded(x):
    """The values that x's MXFP4 form stands for, in 32 bits: each block of 32 columns has the scale 2^e, e = floor(log2 of
    its largest magnitude) - 2, and each value goes to the nearest code (ties to the even one; at most 6)."""
    rows, K = x.shape
    kb = (K + 31) // 32
    b = torch.zeros((rows, 32 * kb), dtype=torch.float32, device=x.device)
    b[:, :K] = x
    b = b.view(rows, kb, 32)
    e = (torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 3).clamp(min=-126)
    v = b.abs() * torch.exp2(-e.float())
    code = (v > 0.25).int() + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5)
    return (_magnitudes(code) * torch.exp2(e.float()) * torch.sign(b)).view(rows, 32 * kb)[:, :K]


def _scales_by_row(scales, rows, kb):
    """Scale bytes of (..., row block, scale block, row mod 32, row / 32 mod 4, scale mod 4) as (..., rows, kb)."""
    s = scales.transpose(-4, -3).transpose(-3, -2).transpose(-4, -3)  # row block, row / 32, row mod 32, scale block, scale
    return s.reshape(scales.shape[:-5] + (128 * scales.shape[-5], 4 * scales.shape[-4]))[..., :rows, :kb]


def _weights(codes, scales):
    """The values that MXFP4 weights stand for, in 32 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).int()
    v = _magnitudes(c & 7) * (1 - 2 * (c >> 3))
    kb = codes.shape[-1] // 16
    s = torch.exp2(_scales_by_row(scales, codes.shape[-2], kb).float() - 127)
    return (v.view(codes.shape[:-1] + (kb, 32)) * s[..., None]).flatten(-2)


def _plain(state):
    op, t, X = state["op"], state["type"], state["X"]
    if op == "quantize":
        return _rounded(X).to(t)
    if op == "linear":
        W = _weights(state["codes"], state["scales"])
        return (_rounded(X) @ W[:, : X.shape[1]].T).to(t)
    o, most, T = state["offsets"], state["most"], X.shape[0]
    if op == "experts":
        W = _weights(state["codes"], state["scales"])[..., : X.shape[1]]
        return _by_row(_by_expert(_rounded(X), o, most) @ W.mT, o, T).to(t)
    W, x = state["W"].float(), _by_expert(X, o, most)
    if op == "forward":
        return _by_row(x @ W, o, T).to(t)
    dy = _by_expert(state["dY"], o, most)
    return {"dX": _by_row(dy @ W.mT, o, T).to(t), "dW": (x.mT @ dy).to(t)}


# ------------------------------------------------------------------ the library's entry points


def _library(state):
    import dense_fp32_gemm_f32_gb300 as g

    op, t, X = state["op"], state["type"], state["X"]
    if op == "forward":
        return g.sgemm_grouped(X, state["W"], state["offsets"])
    if op == "gradient":
        dX = g.sgemm_grouped(state["dY"], state["W"], state["offsets"], transw=True)
        return {"dX": dX, "dW": g.sgemm_grouped_wgrad(X, state["dY"], state["offsets"])}
    if op == "quantize":
        codes, scales = g.sgemm_mxfp4_quantize(X)
        return g.sgemm_mxfp4_dequantize(codes, scales, cols=X.shape[1], dtype=t)
    if op == "linear":
        codes, scales = g.sgemm_mxfp4_quantize(X)
        return g.sgemm_mxfp4(codes, scales, state["codes"], state["scales"], dtype=t)
    codes, scales = g.sgemm_mxfp4_quantize(X, state["offsets"])
    return g.sgemm_mxfp4_grouped(codes, scales, state["codes"], state["scales"], state["offsets"], dtype=t)


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _exact_rounded(x):
    """MXFP4 values of x: for each value the nearest of the grid's, times the block's power of two; ties to even codes."""
    x = x.double()
    out = torch.empty_like(x)
    for k in range(0, x.shape[1], 32):
        b = x[:, k: k + 32]
        m = b.abs().max(1, keepdim=True).values
        s = torch.exp2(((m.view(torch.int64) >> 52) - 1025).clamp(min=-127).double())  # (a double's exponent field, less bias and 2)
        u = b.abs() / s
        best, near = torch.full_like(u, math.inf), torch.zeros_like(u)
        for code in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: an odd one has to be strictly nearer
            d = (u - GRID[code]).abs()
            near = torch.where(d < best, GRID[code], near)
            best = torch.minimum(best, d)
        out[:, k: k + 32] = torch.copysign(near * s, b)
    return out


def _exact_weights(c, s, K):
    """The 4-bit weights (N x K) of one matrix: value of row n, column k from its code and its scale's place."""
    n = torch.arange(c.shape[0], device=c.device)[:, None]
    k = torch.arange(K, device=c.device)[None, :]
    b = k // 32
    scale = torch.exp2(s[n // 128, b // 4, n % 32, (n % 128) // 32, b % 4].double() - 127)
    v = ((c[n, k // 2].int() >> (4 * (k % 2))) & 15).long()
    grid = torch.tensor(GRID + tuple(-u for u in GRID), dtype=torch.float64, device=c.device)
    return grid[v] * scale


def exact(case, seed):
    state = prepare(case, seed)
    op, X = case["op"], state["X"]
    if op == "quantize":
        return _exact_rounded(X)
    if op == "linear":
        return _exact_rounded(X) @ _exact_weights(state["codes"], state["scales"], case["K"]).T
    o = state["offsets"].tolist()
    x = _exact_rounded(X) if op == "experts" else X.double()
    if op == "gradient":
        dX = torch.zeros((case["T"], case["K"]), dtype=torch.float64, device="cuda")
        dW = torch.zeros((case["E"], case["K"], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            dy = state["dY"][o[e]: o[e + 1]].double()
            dX[o[e]: o[e + 1]] = dy @ state["W"][e].double().T
            dW[e] = x[o[e]: o[e + 1]].T @ dy
        return {"dX": dX, "dW": dW}
    Y = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        W = _exact_weights(state["codes"][e], state["scales"][e], case["K"]).T if op == "experts" else state["W"][e].double()
        Y[o[e]: o[e + 1]] = x[o[e]: o[e + 1]] @ W
    return Y
