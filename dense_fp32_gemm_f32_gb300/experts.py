"""Products grouped by expert, and 4-bit microscaled (MXFP4) operands.

Thin binding over include/sgemm_experts.h, which defines the operations, the
layout of MXFP4 operands and the accuracy.  ``offsets`` is an int32 CUDA tensor of E + 1 row boundaries;
it is never read on the host, so no call here waits for the GPU.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib

_TYPES = {torch.float32: _lib.TYPE_F32, torch.bfloat16: _lib.TYPE_BF16, torch.float16: _lib.TYPE_F16}


def _type(dtype, name: str) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return t


def _cuda(X, name: str, dims, dtype=None) -> None:
    if not isinstance(X, torch.Tensor) or not X.is_cuda or (dtype is not None and X.dtype != dtype):
        raise TypeError(f"{name} must be a CUDA {dtype or ''} tensor".replace("  ", " "))
    if X.dim() not in dims:
        raise ValueError(f"{name} must be {' or '.join(map(str, dims))}-D, got shape {tuple(X.shape)}")


def _strides(X, name: str):
    """(row stride, matrix stride) of a 2-D or 3-D tensor with unit column stride."""
    shape, st = X.shape, X.stride()
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = st[-2] if shape[-2] > 1 else shape[-1]
    if ld < shape[-1]:
        raise ValueError(f"{name} has overlapping rows")
    se = st[0] if X.dim() == 3 and shape[0] > 1 else ld * shape[-2]
    return ld, se


def _offsets(offsets, device, name="offsets") -> int:
    _cuda(offsets, name, (1,), torch.int32)
    if offsets.device != device:
        raise ValueError(f"{name} is on another device")
    if offsets.numel() < 1 or (offsets.numel() > 1 and offsets.stride(0) != 1):
        raise ValueError(f"{name} must hold E + 1 contiguous boundaries")
    return offsets.numel() - 1


def _same_device(device, **tensors):
    for name, X in tensors.items():
        if X.device != device:
            raise ValueError(f"{name} is on another device")


@contextlib.contextmanager
def _on(device, stream):
    """Makes ``device`` current, and ``stream`` too if given: outputs that a call
    allocates belong to the stream that its kernels run on."""
    if stream is not None:
        with torch.cuda.device(device), torch.cuda.stream(stream):
            yield int(stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            yield int(torch.cuda.current_stream().cuda_stream)


def _out(out, shape, dtype, device, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(out, torch.Tensor) or out.dtype != dtype or out.device != device or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    return out


def sgemm_grouped(X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None, *,
                  transw: bool = False, stream=None) -> torch.Tensor:
    """``out[t] = X[t] @ op(W[e])`` for the rows ``offsets[e] <= t < offsets[e + 1]`` of each expert, zeros for rows of none.

    ``X`` is (T, K), sorted by expert; ``W`` is (E, K, N), or (E, N, K) with ``transw``; all of one type (float32,
    bfloat16, float16).  The gradient of the rows is the same call on the output's gradient with ``transw`` inverted.
    """
    _cuda(X, "X", (2,))
    _cuda(W, "W", (3,), X.dtype)
    t = _type(X.dtype, "X")
    T, K = X.shape
    E, N = W.shape[0], W.shape[1 if transw else 2]
    if W.shape[2 if transw else 1] != K:
        raise ValueError(f"shapes do not multiply: {(T, K)} x op(W) of {tuple(W.shape)}, transw={bool(transw)}")
    _same_device(X.device, W=W)
    if _offsets(offsets, X.device) != E:
        raise ValueError(f"offsets must hold {E + 1} boundaries, got {offsets.numel()}")
    ldx, _ = _strides(X, "X")
    ldw, sw = _strides(W, "W")
    lib = _lib.load()
    with _on(X.device, stream) as s:
        out = _out(out, (T, N), X.dtype, X.device)
        rc = lib.sgemm_grouped(t, int(bool(transw)), T, E, N, K, X.data_ptr(), ldx, W.data_ptr(), ldw, sw,
                               offsets.data_ptr(), out.data_ptr(), _strides(out, "out")[0], s)
    _lib.check(rc, "sgemm_grouped")
    return out


def sgemm_grouped_wgrad(X: torch.Tensor, dY: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None, *,
                        dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """``out[e] = X[rows of e].T @ dY[rows of e]``: the gradient (E, K, N) of every expert's weights.

    ``X`` is (T, K) and ``dY`` (T, N), of one type; ``dtype`` is that type (default) or float32.  For weights stored
    (E, N, K) swap ``X`` and ``dY``.
    """
    _cuda(X, "X", (2,))
    _cuda(dY, "dY", (2,), X.dtype)
    t = _type(X.dtype, "X")
    dtype = dtype if dtype is not None else out.dtype if out is not None else X.dtype
    if dtype not in (X.dtype, torch.float32):
        raise TypeError(f"the gradient's type must be {X.dtype} or float32, got {dtype}")
    (T, K), N = X.shape, dY.shape[1]
    if dY.shape[0] != T:
        raise ValueError(f"X has {T} rows, dY {dY.shape[0]}")
    _same_device(X.device, dY=dY)
    E = _offsets(offsets, X.device)
    lib = _lib.load()
    with _on(X.device, stream) as s:
        out = _out(out, (E, K, N), dtype, X.device)
        ldo, so = _strides(out, "out")
        rc = lib.sgemm_grouped_wgrad(t, _TYPES[dtype], T, E, K, N, X.data_ptr(), _strides(X, "X")[0], dY.data_ptr(),
                                     _strides(dY, "dY")[0], offsets.data_ptr(), out.data_ptr(), ldo, so, s)
    _lib.check(rc, "sgemm_grouped_wgrad")
    return out


def _blocks(rows: int) -> int:
    return (rows + 127) // 128


def sgemm_mxfp4_quantize(X: torch.Tensor, offsets: torch.Tensor | None = None, *, codes: torch.Tensor | None = None,
                         scales: torch.Tensor | None = None, stream=None):
    """``(codes, scales)``: the MXFP4 form of X's rows, blocks of 32 along the last dimension.

    ``X`` is (rows, K), or (E, rows, K) with scale blocks of its own for each matrix.  ``codes`` has X's leading
    dimensions and 16 * ceil(K / 32) bytes a row; ``scales`` is uint8 (..., row blocks, ceil(K / 128), 32, 4, 4).
    With ``offsets`` the rows are grouped by expert, and every expert's rows begin a scale block.
    """
    _cuda(X, "X", (2, 3))
    t = _type(X.dtype, "X")
    if offsets is not None and X.dim() != 2:
        raise ValueError("rows grouped by expert must be 2-D")
    lead, (rows, K) = tuple(X.shape[:-2]), X.shape[-2:]
    batch = lead[0] if lead else 1
    E = _offsets(offsets, X.device) if offsets is not None else 0
    nb = (rows + 127 * min(rows, E)) // 128 if offsets is not None else _blocks(rows)
    ldx, sx = _strides(X, "X")
    lib = _lib.load()
    with _on(X.device, stream) as s:
        codes = _out(codes, lead + (rows, 16 * ((K + 31) // 32)), torch.uint8, X.device, "codes")
        scales = _out(scales, lead + (nb, _blocks(K), 32, 4, 4), torch.uint8, X.device, "scales")
        _contiguous(codes=codes, scales=scales)
        rc = lib.sgemm_mxfp4_quantize(t, batch, rows, K, X.data_ptr(), ldx, sx, E,
                                      offsets.data_ptr() if offsets is not None else None, codes.data_ptr(),
                                      scales.data_ptr(), s)
    _lib.check(rc, "sgemm_mxfp4_quantize")
    return codes, scales


def _contiguous(**tensors):
    for name, X in tensors.items():
        if not X.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _mxfp4(codes, scales, name: str, dims, cols=None, E: int | None = None):
    """Checks an MXFP4 operand; returns its (rows, 32 * blocks or ``cols``)."""
    _cuda(codes, name, dims, torch.uint8)
    _cuda(scales, f"{name}'s scales", (codes.dim() + 3,), torch.uint8)
    _same_device(codes.device, **{f"{name}'s scales": scales})
    _contiguous(**{name: codes, f"{name}'s scales": scales})
    rows, K = codes.shape[-2], 2 * codes.shape[-1]
    if K % 32:
        raise ValueError(f"{name} must have 16 bytes for each block of 32 columns, got rows of {codes.shape[-1]} bytes")
    nb = _blocks(rows) if E is None else (rows + 127 * min(rows, E)) // 128
    shape = tuple(codes.shape[:-2]) + (nb, _blocks(K), 32, 4, 4)
    if tuple(scales.shape) != shape:
        raise ValueError(f"{name}'s scales must have shape {shape}, got {tuple(scales.shape)}")
    if cols is not None:
        if not 0 <= K - cols < 32:
            raise ValueError(f"{name} holds {K - 31 if K else 0} to {K} columns, not {cols}")
        K = cols
    return rows, K


def sgemm_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor | None = None, *,
                           cols: int | None = None, dtype: torch.dtype = torch.float32,
                           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values that MXFP4 codes and scales stand for (``cols`` columns; default all blocks' 32), as ``dtype``;
    ``offsets`` as given to the quantiser, rows of no expert zero."""
    if out is not None:
        dtype = out.dtype
    t = _type(dtype, "dtype")
    _cuda(codes, "codes", (2, 3), torch.uint8)
    E = _offsets(offsets, codes.device) if offsets is not None else 0
    rows, K = _mxfp4(codes, scales, "codes", (2,) if offsets is not None else (2, 3), cols, E if offsets is not None else None)
    batch = codes.shape[0] if codes.dim() == 3 else 1
    lib = _lib.load()
    with _on(codes.device, stream) as s:
        out = _out(out, tuple(codes.shape[:-1]) + (K,), dtype, codes.device)
        ldy, sy = _strides(out, "out")
        rc = lib.sgemm_mxfp4_dequantize(t, batch, rows, K, codes.data_ptr(), scales.data_ptr(), E,
                                        offsets.data_ptr() if offsets is not None else None, out.data_ptr(), ldy, sy, s)
    _lib.check(rc, "sgemm_mxfp4_dequantize")
    return out


def sgemm_mxfp4(A: torch.Tensor, a_scales: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor,
                out: torch.Tensor | None = None, *, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """``A @ B.T`` (M, N) of two MXFP4 matrices, A (M, K) and B (N, K), both quantised along K, as ``dtype``."""
    M, K = _mxfp4(A, a_scales, "A", (2,))
    N, KB = _mxfp4(B, b_scales, "B", (2,))
    if K != KB:
        raise ValueError(f"A's rows hold {K} columns, B's {KB}")
    _same_device(A.device, B=B)
    dtype = out.dtype if out is not None else dtype
    t = _type(dtype, "dtype")
    lib = _lib.load()
    with _on(A.device, stream) as s:
        out = _out(out, (M, N), dtype, A.device)
        rc = lib.sgemm_mxfp4(t, M, N, K, A.data_ptr(), a_scales.data_ptr(), B.data_ptr(), b_scales.data_ptr(),
                             out.data_ptr(), _strides(out, "out")[0], s)
    _lib.check(rc, "sgemm_mxfp4")
    return out


def sgemm_mxfp4_grouped(X: torch.Tensor, x_scales: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor,
                        offsets: torch.Tensor, out: torch.Tensor | None = None, *,
                        dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """``out[t] = X[t] @ W[e].T`` for the rows of each expert, zeros for rows of none: X (T, K) quantised with the
    same ``offsets``, W (E, N, K) quantised along K."""
    _cuda(X, "X", (2,), torch.uint8)
    E = _offsets(offsets, X.device)
    T, K = _mxfp4(X, x_scales, "X", (2,), E=E)
    N, KW = _mxfp4(W, w_scales, "W", (3,))
    if K != KW or W.shape[0] != E:
        raise ValueError(f"X (columns {K}, {E} experts) and W ({tuple(W.shape)} bytes) do not match")
    _same_device(X.device, W=W)
    dtype = out.dtype if out is not None else dtype
    t = _type(dtype, "dtype")
    lib = _lib.load()
    with _on(X.device, stream) as s:
        out = _out(out, (T, N), dtype, X.device)
        rc = lib.sgemm_mxfp4_grouped(t, T, E, N, K, X.data_ptr(), x_scales.data_ptr(), W.data_ptr(),
                                     w_scales.data_ptr(), offsets.data_ptr(), out.data_ptr(),
                                     _strides(out, "out")[0], s)
    _lib.check(rc, "sgemm_mxfp4_grouped")
    return out
