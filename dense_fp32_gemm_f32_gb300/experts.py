"""Products grouped by expert, and 4-bit microscaled (MXFP4) operands.

Thin binding over include/sgemm_experts.h, which defines the operations, the
layout of MXFP4 operands and the accuracy.  ``offsets`` is an int32 CUDA tensor of E + 1 row boundaries;
it is never read on the host, so no call here waits for the GPU.

As with the library's other entries, results are detached: torch does not differentiate through a call, also where an
operand requires a gradient.  A layer calls the gradients itself, from a torch.autograd.Function around the product
(examples/expert_layer.py has one).
"""
from __future__ import annotations

import torch

from . import _lib

_TYPES = {torch.float32: _lib.TYPE_F32, torch.bfloat16: _lib.TYPE_BF16, torch.float16: _lib.TYPE_F16}


def _type(dtype, name: str) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return t


# A call's host time is what a small product costs, and questions to tensors are
# most of it.  So every function first asks, all at once, whether it has the
# usual call before it: matching CUDA tensors with unit column stride on the
# current device, no `out`, no `stream` (2 us less of 12).  Anything else goes
# the general way, where each check has its message.


def _operand(X, name: str, dim: int, dtype=None):
    """Checks that X is a CUDA tensor of `dim` dimensions (and `dtype`); returns its device's number and its shape."""
    if not isinstance(X, torch.Tensor) or (dtype is not None and X.dtype is not dtype):
        raise TypeError(f"{name} must be a CUDA tensor" + (f" of {dtype}" if dtype is not None else ""))
    dev, shape = X.get_device(), X.shape
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor, got one on {X.device}")
    if len(shape) != dim:
        raise ValueError(f"{name} must be {dim}-D, got shape {tuple(shape)}")
    return dev, shape


def _strides(X, shape, name: str):
    """(row stride, matrix stride) of a 2-D or 3-D tensor with unit column stride."""
    st = X.stride()
    cols, rows = shape[-1], shape[-2]
    if cols > 1 and st[-1] != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = st[-2] if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{name} has overlapping rows")
    return ld, st[0] if len(shape) == 3 and shape[0] > 1 else ld * rows


def _offsets(offsets, dev: int) -> int:
    """Checks the boundaries; returns the number of experts."""
    other, shape = _operand(offsets, "offsets", 1, torch.int32)
    _same_device(dev, other, "offsets")
    n = shape[0]
    if n < 1 or (n > 1 and offsets.stride(0) != 1):
        raise ValueError("offsets must hold E + 1 contiguous boundaries")
    return n - 1


def _same_device(dev: int, other: int, name: str) -> None:
    if other != dev:
        raise ValueError(f"{name} is on another device")


_current_device = torch.cuda.current_device
_empty = torch.empty
_int32, _uint8 = torch.int32, torch.uint8

# The current stream's handle without a Stream object around it, where this torch has that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class _Switch:
    """The operands' device made current, and ``stream`` too if one is given: outputs that a call allocates then belong to
    the stream that its kernels run on.  Undone by close()."""

    def __init__(self, dev: int, stream):
        self.context = torch.cuda.device(dev) if stream is None else torch.cuda.stream(stream)  # (its device too)
        self.context.__enter__()
        if torch.cuda.current_device() != dev:
            self.close()
            raise ValueError("stream is on another device than the operands")

    def close(self):
        self.context.__exit__(None, None, None)


def _enter(dev: int, stream, *tensors):
    """(stream handle, what to close after the call or None).  Nothing is switched in the usual case, the current device
    and stream: a switch costs as much as a launch.  With a ``stream`` the call's tensors (or None) are recorded on it, so
    that the memory of one that the caller drops is not handed out again before the kernels have read it."""
    if stream is None:
        return _raw_stream(dev), (None if torch.cuda.current_device() == dev else _Switch(dev, None))
    switch = _Switch(dev, stream)
    try:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    except BaseException:
        switch.close()
        raise
    return int(stream.cuda_stream), switch


def _out(out, like, shape, dtype, name="out"):
    """(the output, its row stride): allocated beside `like`, or checked."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device), shape[-1]  # (like.new_empty takes 3 us longer)
    if (not isinstance(out, torch.Tensor) or out.dtype != dtype or out.get_device() != like.get_device()
            or tuple(out.shape) != shape):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {shape} on {like.device}")
    return out, _strides(out, shape, name)[0]


def sgemm_grouped(X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None, *,
                  transw: bool = False, stream=None) -> torch.Tensor:
    """``out[t] = X[t] @ op(W[e])`` for the rows ``offsets[e] <= t < offsets[e + 1]`` of each expert, zeros for rows of none.

    ``X`` is (T, K), sorted by expert; ``W`` is (E, K, N), or (E, N, K) with ``transw``; all of one type (float32,
    bfloat16, float16).  The gradient of the rows is the same call on the output's gradient with ``transw`` inverted.
    """
    if out is None and stream is None:
        try:
            dtype, dev, xs, ws, (ldx, ux), (sw, ldw, uw) = X.dtype, X.get_device(), X.shape, W.shape, X.stride(), W.stride()
            t, E, K, N = _TYPES[dtype], ws[0], ws[2 if transw else 1], ws[1 if transw else 2]
            usual = (ux == 1 and uw == 1 and ldx >= K == xs[1] and ldw >= ws[2] and dev >= 0 and W.dtype is dtype
                     and offsets.dtype is _int32 and W.get_device() == dev and offsets.get_device() == dev
                     and offsets.shape == (E + 1,) and offsets.is_contiguous() and _current_device() == dev)
        except (AttributeError, ValueError, KeyError, IndexError):
            usual = False
        if usual:
            T = xs[0]
            out = _empty((T, N), dtype=dtype, device=X.device)
            rc = _lib.load().sgemm_grouped(t, 1 if transw else 0, T, E, N, K, X.data_ptr(), ldx, W.data_ptr(), ldw, sw,
                                           offsets.data_ptr(), out.data_ptr(), N, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_grouped")
            return out
    dev, (T, K) = _operand(X, "X", 2)
    dtype = X.dtype
    t = _type(dtype, "X")
    other, ws = _operand(W, "W", 3, dtype)
    _same_device(dev, other, "W")
    E, N, KW = (ws[0], ws[1], ws[2]) if transw else (ws[0], ws[2], ws[1])
    if KW != K:
        raise ValueError(f"shapes do not multiply: {(T, K)} x op(W) of {tuple(ws)}, transw={bool(transw)}")
    if _offsets(offsets, dev) != E:
        raise ValueError(f"offsets must hold {E + 1} boundaries, got {offsets.numel()}")
    ldx = _strides(X, (T, K), "X")[0]
    ldw, sw = _strides(W, ws, "W")
    s, switch = _enter(dev, stream, X, W, offsets, out)
    try:
        out, ldy = _out(out, X, (T, N), dtype)
        rc = _lib.load().sgemm_grouped(t, 1 if transw else 0, T, E, N, K, X.data_ptr(), ldx, W.data_ptr(), ldw, sw,
                                       offsets.data_ptr(), out.data_ptr(), ldy, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_grouped")
    return out


def sgemm_grouped_wgrad(X: torch.Tensor, dY: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None, *,
                        dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """``out[e] = X[rows of e].T @ dY[rows of e]``: the gradient (E, K, N) of every expert's weights.

    ``X`` is (T, K) and ``dY`` (T, N), of one type; ``dtype`` is that type (default) or float32.  For weights stored
    (E, N, K) swap ``X`` and ``dY``.
    """
    if out is None and stream is None and dtype is None:
        try:
            kind, dev, (T, K), (rows, N), (ldx, ux), (ldy, uy) = X.dtype, X.get_device(), X.shape, dY.shape, X.stride(), dY.stride()
            t, (bounds,) = _TYPES[kind], offsets.shape
            usual = (ux == 1 and uy == 1 and ldx >= K and ldy >= N and rows == T and dev >= 0 and dY.dtype is kind
                     and offsets.dtype is _int32 and dY.get_device() == dev and offsets.get_device() == dev and bounds > 0
                     and offsets.is_contiguous() and _current_device() == dev)
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            out = _empty((bounds - 1, K, N), dtype=kind, device=X.device)
            rc = _lib.load().sgemm_grouped_wgrad(t, t, T, bounds - 1, K, N, X.data_ptr(), ldx, dY.data_ptr(), ldy,
                                                 offsets.data_ptr(), out.data_ptr(), N, K * N, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_grouped_wgrad")
            return out
    dev, (T, K) = _operand(X, "X", 2)
    other, (rows, N) = _operand(dY, "dY", 2, X.dtype)
    _same_device(dev, other, "dY")
    t = _type(X.dtype, "X")
    dtype = dtype if dtype is not None else out.dtype if out is not None else X.dtype
    if dtype not in (X.dtype, torch.float32):
        raise TypeError(f"the gradient's type must be {X.dtype} or float32, got {dtype}")
    if rows != T:
        raise ValueError(f"X has {T} rows, dY {rows}")
    E = _offsets(offsets, dev)
    ldx, ldy = _strides(X, (T, K), "X")[0], _strides(dY, (T, N), "dY")[0]
    s, switch = _enter(dev, stream, X, dY, offsets, out)
    try:
        so = K * N if out is None else None
        out, ldo = _out(out, X, (E, K, N), dtype)
        if so is None:
            so = _strides(out, (E, K, N), "out")[1]
        rc = _lib.load().sgemm_grouped_wgrad(t, _TYPES[dtype], T, E, K, N, X.data_ptr(), ldx, dY.data_ptr(), ldy,
                                             offsets.data_ptr(), out.data_ptr(), ldo, so, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_grouped_wgrad")
    return out


def _grouped_blocks(rows: int, E: int) -> int:
    return (rows + 127 * min(rows, E)) // 128


def sgemm_mxfp4_quantize(X: torch.Tensor, offsets: torch.Tensor | None = None, *, codes: torch.Tensor | None = None,
                         scales: torch.Tensor | None = None, stream=None):
    """``(codes, scales)``: the MXFP4 form of X's rows, blocks of 32 along the last dimension.

    ``X`` is (rows, K), or (E, rows, K) with scale blocks of its own for each matrix.  ``codes`` has X's leading
    dimensions and 16 * ceil(K / 32) bytes a row; ``scales`` is uint8 (..., row blocks, ceil(K / 128), 32, 4, 4).
    With ``offsets`` the rows are grouped by expert, and every expert's rows begin a scale block.
    """
    if codes is None and scales is None and stream is None:
        try:
            t, dev, (rows, K), (ldx, ux) = _TYPES[X.dtype], X.get_device(), X.shape, X.stride()
            usual = ux == 1 and ldx >= K and dev >= 0 and _current_device() == dev
            E, nb, bounds = 0, (rows + 127) // 128, None
            if offsets is not None:
                E = offsets.shape[0] - 1
                nb, bounds = _grouped_blocks(rows, E), offsets.data_ptr()
                usual = (usual and offsets.dtype is _int32 and offsets.get_device() == dev and E >= 0
                         and offsets.dim() == 1 and offsets.is_contiguous())
        except (AttributeError, ValueError, KeyError, IndexError):
            usual = False
        if usual:
            device = X.device
            codes = _empty((rows, 16 * ((K + 31) // 32)), dtype=_uint8, device=device)
            scales = _empty((nb, (K + 127) // 128, 32, 4, 4), dtype=_uint8, device=device)
            rc = _lib.load().sgemm_mxfp4_quantize(t, 1, rows, K, X.data_ptr(), ldx, 0, E, bounds, codes.data_ptr(),
                                                  scales.data_ptr(), _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_mxfp4_quantize")
            return codes, scales
    dim = 3 if isinstance(X, torch.Tensor) and X.dim() == 3 else 2
    dev, shape = _operand(X, "X", dim)
    t = _type(X.dtype, "X")
    rows, K = shape[-2:]
    lead = () if dim == 2 else (shape[0],)
    E, nb = 0, (rows + 127) // 128
    if offsets is not None:
        if dim != 2:
            raise ValueError("rows grouped by expert must be 2-D")
        E = _offsets(offsets, dev)
        nb = _grouped_blocks(rows, E)
    ldx, sx = _strides(X, shape, "X")
    s, switch = _enter(dev, stream, X, offsets, codes, scales)
    try:
        given = codes is not None or scales is not None
        codes, _ = _out(codes, X, lead + (rows, 16 * ((K + 31) // 32)), torch.uint8, "codes")
        scales, _ = _out(scales, X, lead + (nb, (K + 127) // 128, 32, 4, 4), torch.uint8, "scales")
        if given:
            _contiguous(codes, "codes")
            _contiguous(scales, "scales")
        rc = _lib.load().sgemm_mxfp4_quantize(t, shape[0] if dim == 3 else 1, rows, K, X.data_ptr(), ldx, sx, E,
                                              None if offsets is None else offsets.data_ptr(), codes.data_ptr(),
                                              scales.data_ptr(), s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_mxfp4_quantize")
    return codes, scales


def _contiguous(X, name: str) -> None:
    if not X.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _mxfp4(codes, scales, name: str, dim: int, E: int | None = None):
    """Checks an MXFP4 operand (rows grouped by E experts if E is given); returns (device, rows, 32 * blocks)."""
    dev, shape = _operand(codes, name, dim, torch.uint8)
    other, got = _operand(scales, "scales", dim + 3, torch.uint8)
    _same_device(dev, other, "scales")
    _contiguous(codes, name)
    _contiguous(scales, "scales")
    rows, K = shape[-2], 2 * shape[-1]
    if K % 32:
        raise ValueError(f"{name} must have 16 bytes for each block of 32 columns, got rows of {shape[-1]} bytes")
    want = ((rows + 127) // 128 if E is None else _grouped_blocks(rows, E), (K + 127) // 128, 32, 4, 4)
    if got[-5:] != want or got[:-5] != shape[:-2]:
        raise ValueError(f"{name}'s scales must have shape {tuple(shape[:-2]) + want}, got {tuple(got)}")
    return dev, rows, K


def sgemm_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor | None = None, *,
                           cols: int | None = None, dtype: torch.dtype = torch.float32,
                           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values that MXFP4 codes and scales stand for (``cols`` columns; default all blocks' 32), as ``dtype``;
    ``offsets`` as given to the quantiser, rows of no expert zero."""
    if out is None and stream is None and offsets is None:
        try:
            t, dev, (rows, bytes_) = _TYPES[dtype], codes.get_device(), codes.shape
            K = 2 * bytes_ if cols is None else cols
            usual = (not bytes_ % 16 and 0 <= 2 * bytes_ - K < 32 and dev >= 0
                     and _usual_mxfp4(codes, scales, dev, ((rows + 127) // 128, (2 * bytes_ + 127) // 128, 32, 4, 4))
                     and _current_device() == dev)
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            out = _empty((rows, K), dtype=dtype, device=codes.device)
            rc = _lib.load().sgemm_mxfp4_dequantize(t, 1, rows, K, codes.data_ptr(), scales.data_ptr(), 0, None,
                                                    out.data_ptr(), K, 0, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_mxfp4_dequantize")
            return out
    if out is not None:
        dtype = out.dtype
    t = _type(dtype, "dtype")
    dim = 3 if isinstance(codes, torch.Tensor) and codes.dim() == 3 and offsets is None else 2
    E = None if offsets is None else _offsets(offsets, _operand(codes, "codes", 2, torch.uint8)[0])
    dev, rows, K = _mxfp4(codes, scales, "codes", dim, E)
    if cols is not None:
        if not 0 <= K - cols < 32:
            raise ValueError(f"codes hold {max(K - 31, 0)} to {K} columns, not {cols}")
        K = cols
    shape = tuple(codes.shape[:-1]) + (K,)

    s, switch = _enter(dev, stream, codes, scales, offsets, out)
    try:
        sy = rows * K if out is None else None
        out, ldy = _out(out, codes, shape, dtype)
        if sy is None:
            sy = _strides(out, shape, "out")[1]
        rc = _lib.load().sgemm_mxfp4_dequantize(t, shape[0] if dim == 3 else 1, rows, K, codes.data_ptr(), scales.data_ptr(),
                                                E or 0, None if offsets is None else offsets.data_ptr(),
                                                out.data_ptr(), ldy, sy, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_mxfp4_dequantize")
    return out


def _usual_mxfp4(codes, scales, dev: int, shape) -> bool:
    """Whether an MXFP4 operand is as it should be; `shape` of its scales."""
    return (codes.dtype is _uint8 and scales.dtype is _uint8 and codes.get_device() == dev and scales.get_device() == dev
            and scales.shape == shape and codes.is_contiguous() and scales.is_contiguous())


def sgemm_mxfp4(A: torch.Tensor, a_scales: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor,
                out: torch.Tensor | None = None, *, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """``A @ B.T`` (M, N) of two MXFP4 matrices, A (M, K) and B (N, K), both quantised along K, as ``dtype``."""
    if out is None and stream is None:
        try:
            t, dev, (M, bytes_), (N, other) = _TYPES[dtype], A.get_device(), A.shape, B.shape
            kq = (2 * bytes_ + 127) // 128
            usual = (bytes_ == other and not bytes_ % 16 and dev >= 0
                     and _usual_mxfp4(A, a_scales, dev, ((M + 127) // 128, kq, 32, 4, 4))
                     and _usual_mxfp4(B, b_scales, dev, ((N + 127) // 128, kq, 32, 4, 4)) and _current_device() == dev)
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            out = _empty((M, N), dtype=dtype, device=A.device)
            rc = _lib.load().sgemm_mxfp4(t, M, N, 2 * bytes_, A.data_ptr(), a_scales.data_ptr(), B.data_ptr(),
                                         b_scales.data_ptr(), out.data_ptr(), N, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_mxfp4")
            return out
    dev, M, K = _mxfp4(A, a_scales, "A", 2)
    other, N, KB = _mxfp4(B, b_scales, "B", 2)
    _same_device(dev, other, "B")
    if K != KB:
        raise ValueError(f"A's rows hold {K} columns, B's {KB}")
    dtype = out.dtype if out is not None else dtype
    t = _type(dtype, "dtype")

    s, switch = _enter(dev, stream, A, a_scales, B, b_scales, out)
    try:
        out, ldc = _out(out, A, (M, N), dtype)
        rc = _lib.load().sgemm_mxfp4(t, M, N, K, A.data_ptr(), a_scales.data_ptr(), B.data_ptr(), b_scales.data_ptr(),
                                     out.data_ptr(), ldc, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_mxfp4")
    return out


def sgemm_mxfp4_grouped(X: torch.Tensor, x_scales: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor,
                        offsets: torch.Tensor, out: torch.Tensor | None = None, *,
                        dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """``out[t] = X[t] @ W[e].T`` for the rows of each expert, zeros for rows of none: X (T, K) quantised with the
    same ``offsets``, W (E, N, K) quantised along K."""
    if out is None and stream is None:
        try:
            t, dev, (T, bytes_), (E, N, other) = _TYPES[dtype], X.get_device(), X.shape, W.shape
            kq = (2 * bytes_ + 127) // 128
            usual = (bytes_ == other and not bytes_ % 16 and dev >= 0 and offsets.dtype is _int32
                     and offsets.get_device() == dev and offsets.shape == (E + 1,) and offsets.is_contiguous()
                     and _usual_mxfp4(X, x_scales, dev, (_grouped_blocks(T, E), kq, 32, 4, 4))
                     and _usual_mxfp4(W, w_scales, dev, (E, (N + 127) // 128, kq, 32, 4, 4)) and _current_device() == dev)
        except (AttributeError, ValueError, KeyError):
            usual = False
        if usual:
            out = _empty((T, N), dtype=dtype, device=X.device)
            rc = _lib.load().sgemm_mxfp4_grouped(t, T, E, N, 2 * bytes_, X.data_ptr(), x_scales.data_ptr(), W.data_ptr(),
                                                 w_scales.data_ptr(), offsets.data_ptr(), out.data_ptr(), N, _raw_stream(dev))
            if rc:
                _lib.check(rc, "sgemm_mxfp4_grouped")
            return out
    E = _offsets(offsets, _operand(X, "X", 2, torch.uint8)[0])
    dev, T, K = _mxfp4(X, x_scales, "X", 2, E)
    other, N, KW = _mxfp4(W, w_scales, "W", 3)
    _same_device(dev, other, "W")
    if K != KW or W.shape[0] != E:
        raise ValueError(f"X (columns {K}, {E} experts) and W ({tuple(W.shape)} bytes) do not match")
    dtype = out.dtype if out is not None else dtype
    t = _type(dtype, "dtype")

    s, switch = _enter(dev, stream, X, x_scales, W, w_scales, offsets, out)
    try:
        out, ldy = _out(out, X, (T, N), dtype)
        rc = _lib.load().sgemm_mxfp4_grouped(t, T, E, N, K, X.data_ptr(), x_scales.data_ptr(), W.data_ptr(),
                                             w_scales.data_ptr(), offsets.data_ptr(), out.data_ptr(), ldy, s)
    finally:
        if switch is not None:
            switch.close()
    _lib.check(rc, "sgemm_mxfp4_grouped")
    return out
