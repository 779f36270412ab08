"""Orthogonalised weight updates.

Thin binding over include/sgemm_ortho.h, which defines the operation and its accuracy.
"""
from __future__ import annotations

import torch

from . import _lib
from .experts import _TYPES, _current_device, _empty, _enter, _operand, _out, _raw_stream, _strides, _type, _uint8

QUINTIC = (3.4445, -4.7750, 2.0315)


def _quick(t: int, quick: bool) -> int:
    if quick and t != _lib.TYPE_BF16:
        raise ValueError("quick products are for bfloat16 alone")
    return t + _lib.ORTHO_QUICK if quick else t


def _scratch(lib, t: int, E: int, M: int, N: int, steps: int, device):
    """The call's scratch from torch's allocator, on the current stream, to which it goes back when the call has been
    enqueued; (None, 0) where there is none (sizes that the entry refuses among them)."""
    n = lib.sgemm_orthogonalize_workspace(t, E, M, N, steps)
    return (_empty((n,), dtype=_uint8, device=device), n) if n > 0 else (None, 0)


def sgemm_orthogonalize(G: torch.Tensor, out: torch.Tensor | None = None, *, steps: int = 5,
                        coefficients: tuple[float, float, float] = QUINTIC, eps: float = 1e-7, quick: bool = False,
                        stream=None) -> torch.Tensor:
    """``G`` (M, N), or each matrix of (E, M, N) such as sgemm_grouped_wgrad's, with its singular values brought near 1.

    X = G / (|G| + eps), then ``steps`` times X = a X + (b A + c A A) X with A = X X^T (or X^T X, the smaller) and (a, b, c)
    the ``coefficients``: each singular value s becomes a s + b s^3 + c s^5.  The default brings all that are above about
    1/500 of the norm to between 0.7 and 1.2 in five steps; (2, -1.5, 0.5) converges to 1.  M and N are up to 262144.

    Products are as exact as float32's whatever the type, and the result is rounded once.  ``quick``, for bfloat16 alone: a third
    of the work, with operands of 11 bits (4e-4 to 8e-4 of the norm off for the default, as long as G's rank is not low; sgemm_ortho.h says more).
    """
    a, b, c = coefficients
    if out is None and stream is None:
        try:
            t, dev, shape = _TYPES[G.dtype], G.get_device(), G.shape
            M, N = shape[-2:]
            E = shape[0] if len(shape) == 3 else 1
            usual = (2 <= len(shape) <= 3 and G.is_contiguous() and dev >= 0 and _current_device() == dev)
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            t = _quick(t, quick)
            lib = _lib.load()
            out = _empty(shape, dtype=G.dtype, device=G.device)
            scratch, n = _scratch(lib, t, E, M, N, steps, G.device)
            rc = lib.sgemm_orthogonalize(t, E, M, N, G.data_ptr(), N, M * N, steps, a, b, c, eps, out.data_ptr(), N, M * N,
                                         None if scratch is None else scratch.data_ptr(), n, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_orthogonalize")
            return out
    dim = 3 if isinstance(G, torch.Tensor) and G.dim() == 3 else 2
    dev, shape = _operand(G, "G", dim)
    t = _quick(_type(G.dtype, "G"), quick)
    M, N = shape[-2:]
    E = shape[0] if dim == 3 else 1
    ldg, sg = _strides(G, shape, "G")
    s, switch = _enter(dev, stream, G, out)
    try:
        so = M * N if out is None else None
        out, ldo = _out(out, G, tuple(shape), G.dtype)
        if so is None:
            so = _strides(out, shape, "out")[1]
        lib = _lib.load()
        scratch, n = _scratch(lib, t, E, M, N, steps, G.device)
        rc = lib.sgemm_orthogonalize(t, E, M, N, G.data_ptr(), ldg, sg, steps, a, b, c, eps, out.data_ptr(), ldo, so,
                                     None if scratch is None else scratch.data_ptr(), n, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_orthogonalize")
    return out
