"""Python binding of include/hgemm_adapters.h: the linear layer for the rows of
many requests, each with its low-rank adapter.  Argument marshalling only;
re-exported by the package.

Matrices as in layer.py.  Adapters are two 3-D tensors of X's type: A (G, r, K)
and B (G, N, r) with unit stride along the last axis; `which` (M,) int64 says
which of the G a row takes (outside 0 .. G-1: none).
"""
import ctypes

import torch

from . import lib
from .layer import (_MAX_LD, _ONLY, _WIDE, _call, _device, _i64, _int, _linear_operands, _matrix, _mp, _new_room,
                    _room, _saved, _size, _vector, _vp)

EXPORTS_ADAPTERS = ("hg_linear_adapters", "hg_linear_adapters_workspace_size")


class Adapters(ctypes.Structure):
    """struct hg_adapters."""
    _fields_ = [("which", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("A", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("stride_a", ctypes.c_int64), ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64),
                ("stride_b", ctypes.c_int64), ("count", ctypes.c_int64), ("rank", ctypes.c_int32),
                ("type", ctypes.c_int32)]


lib.hg_linear_adapters.argtypes = [_int, _i64, _i64, _i64, _mp, _mp, _vp, _mp, _mp, _mp, ctypes.POINTER(Adapters), _vp,
                                   _i64, _vp]
lib.hg_linear_adapters.restype = _int
lib.hg_linear_adapters_workspace_size.argtypes = [_i64, _i64, _i64, _i64, _mp, _mp]
lib.hg_linear_adapters_workspace_size.restype = _i64


def _stack(t, name, dtype, dev):
    """(address, row stride, stride from one adapter to the next, shape) of a valid stack of matrices."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D")
    if t.get_device() != dev:
        raise ValueError("all tensors must be on one device")
    (count, rows, cols), (stride, ld, unit) = t.shape, t.stride()
    if t.numel() and cols > 1 and unit != 1:
        raise ValueError(f"{name} needs unit stride along its last axis")
    ld = ld if rows > 1 and t.numel() else max(1, cols)
    if not cols <= ld <= _MAX_LD:
        raise ValueError(f"{name}'s rows overlap or are too far apart (row stride {ld}, {cols} columns)")
    return t.data_ptr(), ld, stride if count > 1 and t.numel() else 0, (count, rows, cols)


def _index(t, name, n, dev):
    if not (isinstance(t, torch.Tensor) and t.dtype == torch.int64 and t.dim() == 1 and t.shape[0] == n
            and t.is_contiguous() and t.get_device() == dev):
        raise ValueError(f"{name} must be a contiguous int64 vector of length {n} on the same device")
    return t.data_ptr()


def linear_adapters_workspace_size(X, W, A) -> int:
    """Bytes of workspace linear_adapters needs for these operands
    (hg_linear_adapters_workspace_size); of A (G, r, K) only the rank is looked at."""
    x, w, M, N, K, dev = _linear_operands(X, W)
    return _size(lib.hg_linear_adapters_workspace_size, "hg_linear_adapters_workspace_size", dev, M, N, K, A.shape[1], x, w)


def linear_adapters_workspace(X, W, A):
    """A workspace for linear_adapters calls on these operands (None if they need none)."""
    return _new_room(linear_adapters_workspace_size(X, W, A), X)


def linear_adapters(X, W, Y, which, A, B, scales=None, bias=None, act: int = 0, residual=None, Z=None, work=None):
    """Y = act(X·Wᵀ + bias + s_g·(X·A_gᵀ)·B_gᵀ) + residual with g = which[row] on
    the current stream; returns Y.

    X, W, Y, bias, act, residual and Z as linear's.  which (M,) int64: each row's
    adapter, outside 0 .. G-1 none; A (G, r, K) and B (G, N, r) of X's type, r at
    most 256; scales (G,) float32 or None (1).  `work`: device tensor of at least
    linear_adapters_workspace_size(X, W, A) bytes (allocated with torch when
    None)."""
    x, w, M, N, K, dev = _linear_operands(X, W)
    y, shape = _matrix(Y, "Y", _WIDE[X.dtype], dev)
    if shape[0] != M or shape[1] != N:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, Y {tuple(shape)}")
    a, lda, sa, (count, rank, k) = _stack(A, "A", X.dtype, dev)
    b, ldb, sb, bshape = _stack(B, "B", X.dtype, dev)
    if k != K or bshape != (count, N, rank):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, A {tuple(A.shape)}, B {tuple(B.shape)}")
    s = _vector(scales, "scales", count, dev) if scales is not None else None
    adapters = Adapters(_index(which, "which", M, dev), s, a, lda, sa, b, ldb, sb, count, rank, x.type)
    r = z = bptr = wptr = None
    wbytes = 0
    if bias is not None:
        bptr = _vector(bias, "bias", N, dev)
    if residual is not None:
        r, rshape = _matrix(residual, "residual", _ONLY[Y.dtype], dev)
        if rshape != shape:
            raise ValueError(f"residual {tuple(rshape)} does not match Y {tuple(shape)}")
    if Z is not None:
        z, zshape = _saved(Z, "Z", X.dtype, dev)
        if zshape != shape:
            raise ValueError(f"Z {tuple(zshape)} does not match Y {tuple(shape)}")
    if work is None:
        work = _new_room(_size(lib.hg_linear_adapters_workspace_size, "hg_linear_adapters_workspace_size", dev, M, N, K,
                               rank, x, w), X)
    if work is not None:
        wptr, wbytes = _room(work, dev)
    _call(lib.hg_linear_adapters, "hg_linear_adapters", dev, int(act), M, N, K, x, w, bptr, r, y, z, adapters, wptr, wbytes)
    return Y
