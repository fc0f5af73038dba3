"""Python binding of include/hgemm_linear.h: the linear layer, its gradient
and the 8-bit checkpoints between the two.  Argument marshalling only, as in
the package's other functions; re-exported by the package.

A matrix is a 2-D device tensor with unit stride along its last axis and rows
that do not overlap.  An 8-bit checkpoint is the pair (codes, scales) of
checkpoint8_empty: codes (M, N) uint8 or float8_e4m3fn, scales
(M, ceil(N / 32)) uint8.  All tensors of a call are on one device; the work is
queued on that device's current stream, and tensors that another stream made
or will reuse are the caller's to order, as with the package's other calls.
"""
import ctypes

import torch

from . import HG_BF16, HG_F16, HG_F32, HgError, _raw_stream, lib

HG_E4M3 = 3
E4M3_BLOCK = 32
_MAX_LD = 1 << 30                        # HG_LINEAR_MAX_LD; the row stride of a single row does not count
ACT_GELU = 2
ACT_GELU_TANH = 3
ACT_SILU = 4

EXPORTS_LINEAR = ("hg_linear", "hg_linear_workspace_size", "hg_linear_grad", "hg_linear_grad_workspace_size",
                  "hg_checkpoint8_write", "hg_checkpoint8_read")


class Matrix(ctypes.Structure):
    """struct hg_matrix."""
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("lds", ctypes.c_int64), ("type", ctypes.c_int32)]


_i64, _vp, _int, _mp = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(Matrix)
lib.hg_linear.argtypes = [_int, _i64, _i64, _i64, _mp, _mp, _vp, _mp, _mp, _mp, _vp, _i64, _vp]
lib.hg_linear.restype = _int
lib.hg_linear_workspace_size.argtypes = [_i64, _i64, _i64, _mp, _mp]
lib.hg_linear_workspace_size.restype = _i64
lib.hg_linear_grad.argtypes = [_int, _i64, _i64, _i64, _mp, _mp, _mp, _mp, _mp, _mp, _vp, _int, _vp, _i64, _vp]
lib.hg_linear_grad.restype = _int
lib.hg_linear_grad_workspace_size.argtypes = [_i64, _i64, _i64, _mp, _mp, _mp]
lib.hg_linear_grad_workspace_size.restype = _i64
lib.hg_checkpoint8_write.argtypes = [_i64, _i64, _mp, _mp, _vp]
lib.hg_checkpoint8_write.restype = _int
lib.hg_checkpoint8_read.argtypes = [_i64, _i64, _mp, _mp, _vp]
lib.hg_checkpoint8_read.restype = _int

# torch's getter of the current device without the checks of
# torch.cuda.current_device() (the tensors at hand are on the GPU already).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream = _raw_stream or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_HALF = {torch.float16: HG_F16, torch.bfloat16: HG_BF16}
_ONLY = {torch.float16: {torch.float16: HG_F16}, torch.bfloat16: {torch.bfloat16: HG_BF16},
         torch.float32: {torch.float32: HG_F32}}
_WIDE = {t: {t: c, torch.float32: HG_F32} for t, c in _HALF.items()}       # a type or float32
_CODES = {torch.uint8: HG_E4M3, torch.float8_e4m3fn: HG_E4M3}
_BYTES = {torch.uint8: HG_E4M3}


def _lead(t, name, types, dev):
    """The leading dimension of a valid matrix on device `dev`; raises for
    anything else."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(types)}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.get_device() != dev:
        raise ValueError("all tensors must be on one device")
    (rows, cols), (ld, unit) = t.shape, t.stride()
    if rows and cols > 1 and unit != 1:
        raise ValueError(f"{name} needs unit stride along its last axis")
    if rows > 1 and cols and ld < cols:
        raise ValueError(f"{name}'s rows overlap (row stride {ld}, {cols} columns)")
    return ld if rows > 1 and cols else max(1, cols)


def _matrix(t, name, types, dev, part=""):
    """(struct hg_matrix, shape)."""
    try:                                 # an ordinary matrix, without the checks that name what is wrong
        ld, unit = t.stride()
        shape = t.shape
        if unit == 1 and _MAX_LD >= ld >= shape[1] > 0 and t.get_device() == dev:
            return Matrix(t.data_ptr(), ld, None, 0, types[t.dtype]), shape
    except (AttributeError, KeyError, TypeError, ValueError):
        pass
    ld = _lead(t, name + part, types, dev)
    return Matrix(t.data_ptr(), ld, None, 0, types[t.dtype]), t.shape


def _pair(pair, name, dev):
    if not (isinstance(pair, (tuple, list)) and len(pair) == 2):
        raise TypeError(f"{name} must be a tensor or a pair (codes, scales)")
    codes, scales = pair
    c, shape = _matrix(codes, name, _CODES, dev, "'s codes")
    s, have = _matrix(scales, name, _BYTES, dev, "'s scales")
    rows, cols = shape
    if have[0] != rows or have[1] != -(-cols // E4M3_BLOCK):
        raise ValueError(f"{name}'s scales {tuple(have)} do not match codes {tuple(shape)}: "
                         f"expected {(rows, -(-cols // E4M3_BLOCK))}")
    c.scales, c.lds = s.data, s.ld
    return c, shape


def _saved(m, name, dtype, dev):
    """(matrix, shape) of a 16-bit tensor or an 8-bit checkpoint."""
    return _matrix(m, name, _ONLY[dtype], dev) if isinstance(m, torch.Tensor) else _pair(m, name, dev)


def _device(t, name):
    try:
        dev = t.get_device()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    return dev if dev >= 0 else None                   # _lead refuses the host's by name


def _vector(v, name, n, dev):
    if not (isinstance(v, torch.Tensor) and v.dtype == torch.float32 and v.dim() == 1 and v.shape[0] == n
            and v.is_contiguous() and v.get_device() == dev):
        raise ValueError(f"{name} must be a contiguous float32 vector of length {n} on the same device")
    return v.data_ptr()


def _room(work, dev):
    """(address, bytes) of a caller's workspace."""
    if not (isinstance(work, torch.Tensor) and work.is_contiguous() and work.get_device() == dev):
        raise ValueError("work must be a contiguous tensor on the same device")
    return work.data_ptr(), work.numel() * work.element_size()


def _new_room(need, like):
    return torch.empty(need, dtype=torch.uint8, device=like.device) if need else None


def _elsewhere(fn, dev, args):
    with torch.cuda.device(dev):
        return fn(*args)


def _call(fn, name, dev, *args):
    """fn(*args, the current stream of device `dev`), with that device current."""
    args += (_stream(dev),)
    st = fn(*args) if _current_device() == dev else _elsewhere(fn, dev, args)
    if st != 0:
        raise HgError(name, st)


def _size(fn, name, dev, *args):
    need = fn(*args) if _current_device() == dev else _elsewhere(fn, dev, args)
    if need < 0:
        raise HgError(name, int(need))
    return int(need)


_NO_WORK = -11              # hg_linear: a workspace is needed and there is none


def _linear_operands(X, W):
    dev = _device(X, "X")
    x, (M, K) = _matrix(X, "X", _HALF, dev)
    w, (N, k) = _matrix(W, "W", _ONLY[X.dtype], dev)
    if k != K:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}")
    return x, w, M, N, K, dev


def linear_workspace_size(X, W) -> int:
    """Bytes of workspace linear needs for these operands (hg_linear_workspace_size)."""
    x, w, M, N, K, dev = _linear_operands(X, W)
    return _size(lib.hg_linear_workspace_size, "hg_linear_workspace_size", dev, M, N, K, x, w)


def linear_workspace(X, W):
    """A workspace for linear calls on these operands (None if they need none)."""
    return _new_room(linear_workspace_size(X, W), X)


def linear(X, W, Y, bias=None, act: int = 0, residual=None, Z=None, work=None):
    """Y = act(X·Wᵀ + bias) + residual on the current stream; returns Y.

    X (M, K) and W (N, K) float16 or bfloat16, Y (M, N) of their type or
    float32, bias a float32 vector of length N, residual (M, N) of Y's type
    (Y itself: in place).  The pre-activation X·Wᵀ + bias is saved in Z, an
    (M, N) tensor of X's type or an 8-bit checkpoint (codes, scales).  `work`:
    device tensor of at least linear_workspace_size(X, W) bytes (allocated with
    torch when None and needed)."""
    x, w, M, N, K, dev = _linear_operands(X, W)
    y, shape = _matrix(Y, "Y", _WIDE[X.dtype], dev)
    if shape[0] != M or shape[1] != N:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, Y {tuple(shape)}")
    r = z = b = wptr = None
    wbytes = 0
    if bias is not None:
        b = _vector(bias, "bias", N, dev)
    if residual is not None:
        r, rshape = _matrix(residual, "residual", _ONLY[Y.dtype], dev)
        if rshape != shape:
            raise ValueError(f"residual {tuple(rshape)} does not match Y {tuple(shape)}")
    if Z is not None:
        z, zshape = _saved(Z, "Z", X.dtype, dev)
        if zshape != shape:
            raise ValueError(f"Z {tuple(zshape)} does not match Y {tuple(shape)}")
    if work is not None:
        wptr, wbytes = _room(work, dev)
    args = (int(act), M, N, K, x, w, b, r, y, z)
    try:
        _call(lib.hg_linear, "hg_linear", dev, *args, wptr, wbytes)
    except HgError as e:
        if work is not None or e.status != _NO_WORK:
            raise
        need = _size(lib.hg_linear_workspace_size, "hg_linear_workspace_size", dev, M, N, K, x, w)
        _call(lib.hg_linear, "hg_linear", dev, *args, _new_room(need, X).data_ptr(), need)
    return Y


def _grad_operands(dY, W, X):
    dev = _device(dY, "dY")
    dy, (M, N) = _matrix(dY, "dY", _HALF, dev)
    w = x = K = None
    if W is not None:
        w, (n, K) = _matrix(W, "W", _ONLY[dY.dtype], dev)
        if n != N:
            raise ValueError(f"shape mismatch: dY {tuple(dY.shape)}, W {tuple(W.shape)}")
    if X is not None:
        x, shape = _saved(X, "X", dY.dtype, dev)
        if shape[0] != M or K not in (None, shape[1]):
            raise ValueError(f"shape mismatch: dY {tuple(dY.shape)}, X {tuple(shape)}"
                             + (f", W {tuple(W.shape)}" if W is not None else ""))
        K = shape[1]
    return dy, w, x, M, N, K or 0, dev


def linear_grad_workspace_size(dY, W, X) -> int:
    """Bytes of workspace linear_grad needs for these operands
    (hg_linear_grad_workspace_size); W or X None: without dX or dW."""
    dy, w, x, M, N, K, dev = _grad_operands(dY, W, X)
    return _size(lib.hg_linear_grad_workspace_size, "hg_linear_grad_workspace_size", dev, M, N, K, dy, w, x)


def linear_grad_workspace(dY, W, X):
    """A workspace for linear_grad calls on these operands."""
    return _new_room(linear_grad_workspace_size(dY, W, X), dY)


def linear_grad(dY, W, X, Z=None, act: int = 0, dX=None, dW=None, dbias=None, accumulate: bool = False, work=None):
    """The gradients of linear on the current stream: dz = dY·act'(Z), dX =
    dz·W, dW = dzᵀ·X, dbias = the column sums of dz; returns (dX, dW, dbias).

    dY (M, N) float16 or bfloat16, W (N, K) of its type, X (M, K) and Z (M, N)
    of its type or 8-bit checkpoints (codes, scales).  Only the gradients that
    are given are computed: dX (M, K) of dY's type, dW (N, K) of dY's type or
    float32, dbias float32 of length N.  W may be None without dX, X without
    dW, Z with ACT_NONE.  `accumulate`: dW and dbias are added to.  dz is
    rounded to dY's type for dX and dW (float16: infinite past 65504).  `work`:
    device tensor of at least linear_grad_workspace_size(dY, W, X) bytes
    (allocated with torch when None)."""
    dy, w, x, M, N, K, dev = _grad_operands(dY, W, X)
    z = gx = gw = gb = wptr = None
    wbytes = 0
    if dX is not None:
        if W is None:
            raise ValueError("dX needs W")
        gx, shape = _matrix(dX, "dX", _ONLY[dY.dtype], dev)
        if shape[0] != M or shape[1] != K:
            raise ValueError(f"dX {tuple(shape)} does not match {(M, K)}")
    if dW is not None:
        if X is None:
            raise ValueError("dW needs X")
        gw, shape = _matrix(dW, "dW", _WIDE[dY.dtype], dev)
        if shape[0] != N or shape[1] != K:
            raise ValueError(f"dW {tuple(shape)} does not match {(N, K)}")
    if dbias is not None:
        gb = _vector(dbias, "dbias", N, dev)
    if Z is not None:
        z, shape = _saved(Z, "Z", dY.dtype, dev)
        if shape[0] != M or shape[1] != N:
            raise ValueError(f"Z {tuple(shape)} does not match dY {(M, N)}")
    elif act != 0:
        raise ValueError("the activation's gradient needs Z")
    if work is None:
        work = _new_room(_size(lib.hg_linear_grad_workspace_size, "hg_linear_grad_workspace_size", dev, M, N, K, dy, w,
                               x), dY)
    if work is not None:
        wptr, wbytes = _room(work, dev)
    _call(lib.hg_linear_grad, "hg_linear_grad", dev, int(act), M, N, K, dy, w, x, z, gx, gw, gb,
          1 if accumulate else 0, wptr, wbytes)
    return dX, dW, dbias


def checkpoint8_empty(M: int, N: int, device="cuda"):
    """Room for the 8-bit checkpoint of an (M, N) matrix: (codes, scales)."""
    return (torch.empty((M, N), dtype=torch.uint8, device=device),
            torch.empty((M, -(-N // E4M3_BLOCK)), dtype=torch.uint8, device=device))


def _checkpoint(X, codes, scales):
    dev = _device(X, "X")
    (x, shape), (c, have) = _matrix(X, "X", _HALF, dev), _pair((codes, scales), "the checkpoint", dev)
    if have != shape:
        raise ValueError(f"codes {tuple(have)} do not match X {tuple(shape)}")
    return x, c, *shape, dev


def checkpoint8_write(X, codes, scales):
    """X (float16 or bfloat16) as an 8-bit checkpoint; returns (codes, scales)."""
    x, c, M, N, dev = _checkpoint(X, codes, scales)
    _call(lib.hg_checkpoint8_write, "hg_checkpoint8_write", dev, M, N, x, c)
    return codes, scales


def checkpoint8_read(codes, scales, X):
    """The values of an 8-bit checkpoint, written to X (float16 or bfloat16); returns X."""
    x, c, M, N, dev = _checkpoint(X, codes, scales)
    _call(lib.hg_checkpoint8_read, "hg_checkpoint8_read", dev, M, N, c, x)
    return X
