"""Routing of tokens to experts, and their rows' way there and back.

Thin binding over include/sgemm_routing.h, which defines the operations.  The results are what the grouped products of
``experts.py`` take: ``offsets`` and rows sorted by expert.  Nothing here waits for the GPU, and results are detached, as
those of the library's other entries: a layer calls the gradients itself (examples/expert_layer.py does).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from .experts import _TYPES, _contiguous, _current_device, _empty, _enter, _int32, _offsets, _operand, _out, _raw_stream, _same_device, _strides, _type

_float32 = torch.float32
_SCORES = {"softmax": _lib.SCORE_SOFTMAX, "sigmoid": _lib.SCORE_SIGMOID}


class Routing(NamedTuple):
    """Every token's choices: ``experts`` (T, k) int32, the best first, -1 where there is none; their ``weights`` (T, k)
    float32; the boundaries of the experts' rows, ``offsets`` (E + 1,) int32; and each choice's row among all choices
    sorted by expert, ``slots`` (T, k) int32."""

    experts: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    slots: torch.Tensor


def _score(score) -> int:
    s = _SCORES.get(score)
    if s is None:
        raise ValueError(f"score must be one of {', '.join(_SCORES)}, got {score!r}")
    return s


def _choices(X, name: str, dev: int, dtype=_int32):
    """Checks a contiguous (T, k) tensor; returns its shape."""
    other, shape = _operand(X, name, 2, dtype)
    _same_device(dev, other, name)
    _contiguous(X, name)
    return shape


def sgemm_route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
                top_groups: int | None = None, group_best: int = 1, renormalize: bool = False, scale: float = 1.0,
                stream=None) -> Routing:
    """The ``k`` experts of each token (row of ``logits``, (T, E)) with the largest score + ``bias``, and their weights.

    ``score`` is "softmax" or "sigmoid" of the logits; ``bias`` (E,) float32 has a part in the choice alone.  With
    ``groups`` the choice is from the ``top_groups`` groups of E / groups neighbours with the largest sum of their
    ``group_best`` (1 or 2) best.  Weights are ``scale`` times the chosen scores, divided by their sum with
    ``renormalize``.  Experts whose logit is -inf are out of service; a row of -inf has no experts (-1, weight 0).
    Ties go to the lowest index.
    """
    top = groups if top_groups is None else top_groups
    if stream is None:
        try:
            t, dev, (T, E), (ld, u) = _TYPES[logits.dtype], logits.get_device(), logits.shape, logits.stride()
            usual = (u == 1 and ld >= E and dev >= 0 and E > 0 and _current_device() == dev
                     and (bias is None or (bias.dtype is _float32 and bias.get_device() == dev and bias.shape == (E,)
                                           and bias.is_contiguous())))
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            return _route(t, _score(score), T, E, k, logits, ld, bias, groups, top, group_best, renormalize, scale, _raw_stream(dev))
    dev, (T, E) = _operand(logits, "logits", 2)
    t = _type(logits.dtype, "logits")
    code = _score(score)
    ld = _strides(logits, (T, E), "logits")[0]
    if E < 1:
        raise ValueError("logits must have a column for each expert")
    if bias is not None:
        other, shape = _operand(bias, "bias", 1, _float32)
        _same_device(dev, other, "bias")
        if tuple(shape) != (E,):
            raise ValueError(f"bias must have shape {(E,)}, got {tuple(shape)}")
        _contiguous(bias, "bias")
    s, switch = _enter(dev, stream, logits, bias)
    try:
        return _route(t, code, T, E, k, logits, ld, bias, groups, top, group_best, renormalize, scale, s)
    finally:
        if switch is not None:
            switch.close()


def _route(t, code, T, E, k, logits, ld, bias, groups, top_groups, group_best, renormalize, scale, s) -> Routing:
    if not 1 <= k <= min(E, 32) or E > 1024:
        raise ValueError(f"a token can have 1 to 32 of at most 1024 experts, not {k} of {E}")
    if not 1 <= groups <= 32 or E % groups or not 1 <= top_groups <= groups or group_best not in (1, 2):
        raise ValueError(f"{E} experts cannot be chosen from {top_groups} of {groups} groups by their {group_best} best")
    device = logits.device
    experts = _empty((T, k), dtype=_int32, device=device)
    weights = _empty((T, k), dtype=_float32, device=device)
    offsets = _empty((E + 1,), dtype=_int32, device=device)
    slots = _empty((T, k), dtype=_int32, device=device)
    rc = _lib.load().sgemm_route(t, code, T, E, k, logits.data_ptr(), ld, None if bias is None else bias.data_ptr(), groups,
                                 top_groups, group_best, 1 if renormalize else 0, scale, experts.data_ptr(), weights.data_ptr(),
                                 offsets.data_ptr(), slots.data_ptr(), s)
    if rc:
        _lib.check(rc, "sgemm_route")
    return Routing(experts, weights, offsets, slots)


def sgemm_route_grad(logits: torch.Tensor, experts: torch.Tensor, dweights: torch.Tensor, out: torch.Tensor | None = None, *,
                     score: str = "softmax", renormalize: bool = False, scale: float = 1.0, stream=None) -> torch.Tensor:
    """The gradient (T, E) of the logits from ``dweights`` (T, k), that of the weights of ``experts`` (T, k) which
    sgemm_route chose with the same ``score``, ``renormalize`` and ``scale``."""
    if out is None and stream is None:
        try:
            t, dev, (T, E), (ld, u), shape = _TYPES[logits.dtype], logits.get_device(), logits.shape, logits.stride(), experts.shape
            usual = (u == 1 and ld >= E and dev >= 0 and _current_device() == dev and len(shape) == 2 and shape[0] == T
                     and 1 <= shape[1] <= E <= 1024 and shape[1] <= 32
                     and experts.dtype is _int32 and dweights.dtype is _float32 and dweights.shape == shape
                     and experts.get_device() == dev and dweights.get_device() == dev and experts.is_contiguous()
                     and dweights.is_contiguous())
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            out = _empty((T, E), dtype=logits.dtype, device=logits.device)
            rc = _lib.load().sgemm_route_grad(t, _score(score), T, E, shape[1], logits.data_ptr(), ld, experts.data_ptr(),
                                              dweights.data_ptr(), 1 if renormalize else 0, scale, out.data_ptr(), E, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_route_grad")
            return out
    dev, (T, E) = _operand(logits, "logits", 2)
    t = _type(logits.dtype, "logits")
    code = _score(score)
    ld = _strides(logits, (T, E), "logits")[0]
    rows, k = _choices(experts, "experts", dev)
    if rows != T or not 1 <= k <= min(E, 32) or E > 1024:
        raise ValueError(f"experts must be ({T}, k) with k from 1 to 32 and at most E <= 1024, got {(rows, k)} and E = {E}")
    if tuple(_choices(dweights, "dweights", dev, _float32)) != (T, k):
        raise ValueError(f"dweights must have the experts' shape {(T, k)}, got {tuple(dweights.shape)}")
    s, switch = _enter(dev, stream, logits, experts, dweights, out)
    try:
        out, ldd = _out(out, logits, (T, E), logits.dtype)
        rc = _lib.load().sgemm_route_grad(t, code, T, E, k, logits.data_ptr(), ld, experts.data_ptr(), dweights.data_ptr(),
                                          1 if renormalize else 0, scale, out.data_ptr(), ldd, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_route_grad")
    return out


def sgemm_spread(X: torch.Tensor, slots: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None, *,
                 stream=None) -> torch.Tensor:
    """``out[slots[t, j]] = X[t]``: every token's row to the places of its choices, zeros to the rows from ``offsets[-1]`` on
    (also to one that a slot names).

    ``X`` is (T, H), ``slots`` (T, k) and ``offsets`` as sgemm_route gives them; ``out`` has T * k rows by default.  Its
    gradient is sgemm_combine of the gradient, without weights.
    """
    if out is None and stream is None:
        try:
            t, dev, (T, H), (ldx, u), (rows, k) = _TYPES[X.dtype], X.get_device(), X.shape, X.stride(), slots.shape
            usual = (u == 1 and ldx >= H and rows == T and dev >= 0 and _current_device() == dev and slots.dtype is _int32
                     and offsets.dtype is _int32 and slots.get_device() == dev and offsets.get_device() == dev
                     and slots.is_contiguous() and offsets.dim() == 1 and offsets.is_contiguous() and offsets.shape[0] > 0)
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            out = _empty((T * k, H), dtype=X.dtype, device=X.device)
            rc = _lib.load().sgemm_spread(t, T, k, T * k, H, X.data_ptr(), ldx, slots.data_ptr(), offsets.shape[0] - 1,
                                          offsets.data_ptr(), out.data_ptr(), H, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_spread")
            return out
    dev, (T, H) = _operand(X, "X", 2)
    t = _type(X.dtype, "X")
    rows, k = _choices(slots, "slots", dev)
    if rows != T:
        raise ValueError(f"X has {T} rows, slots {rows}")
    E = _offsets(offsets, dev)
    ldx = _strides(X, (T, H), "X")[0]
    R = T * k
    if out is not None:
        R = _operand(out, "out", 2, X.dtype)[1][0]
    s, switch = _enter(dev, stream, X, slots, offsets, out)
    try:
        out, ldy = _out(out, X, (R, H), X.dtype)
        rc = _lib.load().sgemm_spread(t, T, k, R, H, X.data_ptr(), ldx, slots.data_ptr(), E, offsets.data_ptr(), out.data_ptr(), ldy, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_spread")
    return out


def sgemm_combine(Y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None, out: torch.Tensor | None = None, *,
                  stream=None) -> torch.Tensor:
    """``out[t] = sum over j of weights[t, j] * Y[slots[t, j]]`` (T, H), choices without a row left out; ``weights`` (T, k)
    float32, default ones."""
    if out is None and stream is None:
        try:
            t, dev, (R, H), (ldy, u), shape = _TYPES[Y.dtype], Y.get_device(), Y.shape, Y.stride(), slots.shape
            T, k = shape
            usual = (u == 1 and ldy >= H and dev >= 0 and _current_device() == dev and slots.dtype is _int32
                     and slots.get_device() == dev and slots.is_contiguous()
                     and (weights is None or (weights.dtype is _float32 and weights.shape == shape and weights.get_device() == dev
                                              and weights.is_contiguous())))
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            out = _empty((T, H), dtype=Y.dtype, device=Y.device)
            rc = _lib.load().sgemm_combine(t, T, k, R, H, Y.data_ptr(), ldy, slots.data_ptr(),
                                           None if weights is None else weights.data_ptr(), out.data_ptr(), H, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_combine")
            return out
    dev, (R, H) = _operand(Y, "Y", 2)
    t = _type(Y.dtype, "Y")
    T, k = _choices(slots, "slots", dev)
    if weights is not None and tuple(_choices(weights, "weights", dev, _float32)) != (T, k):
        raise ValueError(f"weights must have the slots' shape {(T, k)}, got {tuple(weights.shape)}")
    ldy = _strides(Y, (R, H), "Y")[0]
    s, switch = _enter(dev, stream, Y, slots, weights, out)
    try:
        out, ldo = _out(out, Y, (T, H), Y.dtype)
        rc = _lib.load().sgemm_combine(t, T, k, R, H, Y.data_ptr(), ldy, slots.data_ptr(),
                                       None if weights is None else weights.data_ptr(), out.data_ptr(), ldo, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_combine")
    return out


def sgemm_combine_grad(dout: torch.Tensor, Y: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None,
                       offsets: torch.Tensor, *, needs: tuple[bool, bool] = (True, True), stream=None):
    """``(dY, dweights)`` of sgemm_combine from the gradient ``dout`` (T, H) of its result: (R, H) of ``Y``'s type, zeros
    from ``offsets[-1]`` on, and (T, k) float32.  ``needs``: which of the two are wanted; the other is None."""
    dev, (T, H) = _operand(dout, "dout", 2)
    dtype = dout.dtype
    t = _type(dtype, "dout")
    other, (R, HY) = _operand(Y, "Y", 2, dtype)
    _same_device(dev, other, "Y")
    rows, k = _choices(slots, "slots", dev)
    if HY != H or rows != T:
        raise ValueError(f"dout {(T, H)}, Y {(R, HY)} and slots {(rows, k)} do not match")
    if weights is not None and tuple(_choices(weights, "weights", dev, _float32)) != (T, k):
        raise ValueError(f"weights must have the slots' shape {(T, k)}, got {tuple(weights.shape)}")
    E = _offsets(offsets, dev)
    ldd, ldy = _strides(dout, (T, H), "dout")[0], _strides(Y, (R, H), "Y")[0]
    s, switch = _enter(dev, stream, dout, Y, slots, weights, offsets)
    try:
        dY = _empty((R, H), dtype=dtype, device=dout.device) if needs[0] else None
        dweights = _empty((T, k), dtype=_float32, device=dout.device) if needs[1] else None
        rc = _lib.load().sgemm_combine_grad(t, T, k, R, H, dout.data_ptr(), ldd, Y.data_ptr(), ldy, slots.data_ptr(),
                                            None if weights is None else weights.data_ptr(), E, offsets.data_ptr(),
                                            None if dY is None else dY.data_ptr(), H,
                                            None if dweights is None else dweights.data_ptr(), s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_combine_grad")
    return dY, dweights
