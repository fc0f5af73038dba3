"""Python binding of include/hgemm_adamw.h: a step of AdamW over many tensors,
their moments in fp32 or as 8-bit checkpoints.  Argument marshalling only;
re-exported by the package.

A tensor is contiguous, of any shape, and counts as its elements one after the
other.  A moment is a float32 tensor of as many elements, or in 8 bits a pair
(codes, scales) of contiguous tensors of n and ceil(n / 32) bytes, as adamw_state
makes them.  All tensors of a call are on one device.
"""
import ctypes

import torch

from . import HG_F32, lib
from .layer import _CODES, E4M3_BLOCK, HG_E4M3, HgError, _call, _device, _i64, _int, _vp
from .logits import _LOGITS as _FLOATS

EXPORTS_ADAMW = ("hg_adamw", "hg_adamw_check")
_double = ctypes.c_double


class AdamWTensor(ctypes.Structure):
    """struct hg_adamw_tensor."""
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("m_scales", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("n", ctypes.c_int64), ("param_type", ctypes.c_int32),
                ("grad_type", ctypes.c_int32), ("state_type", ctypes.c_int32)]


lib.hg_adamw.argtypes = [_i64, ctypes.POINTER(AdamWTensor), _i64, _vp, _double, _double, _double, _double, _double, _vp,
                         ctypes.c_uint64, _vp]
lib.hg_adamw.restype = _int
lib.hg_adamw_check.argtypes = [_i64, ctypes.POINTER(AdamWTensor)]
lib.hg_adamw_check.restype = _int


def _flat(t, name, types, n, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(types)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError("all tensors must be on one device")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    return t.data_ptr()


def _moment(x, name, n, dev):
    """(address, address of the scales, type)"""
    if isinstance(x, torch.Tensor):
        return _flat(x, name, (torch.float32,), n, dev), None, HG_F32
    if not (isinstance(x, (tuple, list)) and len(x) == 2):
        raise TypeError(f"{name} must be a tensor or a pair (codes, scales)")
    return (_flat(x[0], name + "'s codes", _CODES, n, dev),
            _flat(x[1], name + "'s scales", (torch.uint8,), -(-n // E4M3_BLOCK), dev), HG_E4M3)


class AdamWTensors:
    """The tensors of a program's steps, checked once: adamw_tensors()."""

    def __init__(self, params, grads, m, v, masters=None):
        params, grads, m, v = list(params), list(grads), list(m), list(v)
        masters = [None] * len(params) if masters is None else list(masters)
        if not len(params) == len(grads) == len(m) == len(v) == len(masters):
            raise ValueError("params, grads, m, v and masters must be lists of one length")
        self.held = params, grads, m, v, masters           # the tensors live as long as their addresses are used
        self.count = len(params)
        self.array = (AdamWTensor * max(1, self.count))()
        self.device = _device(params[0], "params[0]") if params else None
        for i, (p, g, a, b, w) in enumerate(zip(params, grads, m, v, masters)):
            if not isinstance(p, torch.Tensor):
                raise TypeError(f"params[{i}] must be a torch.Tensor")
            if not p.is_cuda:
                raise ValueError(f"params[{i}] must be a device tensor")
            n, dev = p.numel(), self.device
            (am, asc, at), (bm, bsc, bt) = _moment(a, f"m[{i}]", n, dev), _moment(b, f"v[{i}]", n, dev)
            if at != bt:
                raise ValueError(f"m[{i}] and v[{i}] must be in the same form")
            master = None
            if w is not None:
                if p.dtype == torch.float32:
                    raise ValueError(f"params[{i}] is float32 and has no master")
                master = _flat(w, f"masters[{i}]", (torch.float32,), n, dev)
            self.array[i] = AdamWTensor(_flat(p, f"params[{i}]", _FLOATS, n, dev), master,
                                        _flat(g, f"grads[{i}]", _FLOATS, n, dev), am, asc, bm, bsc, n, _FLOATS[p.dtype],
                                        _FLOATS[g.dtype], at)
        status = lib.hg_adamw_check(self.count, self.array)
        if status != 0:
            raise HgError("hg_adamw_check", status)


def adamw_tensors(params, grads, m, v, masters=None) -> AdamWTensors:
    """Tensors for adamw, checked once (types, sizes, and that none that is written
    overlaps another) and held: lists of one length.

    params float16, bfloat16 or float32; grads of any of these; m and v float32 or
    pairs (codes, scales), see adamw_state; masters float32 tensors or None in
    places, the weights that 16-bit params are the roundings of."""
    return AdamWTensors(params, grads, m, v, masters)


def adamw_state(param, bits: int = 32):
    """(m, v) of zero for a param: float32 tensors, or with bits = 8 pairs (codes,
    scales).  Codes of a 2-D param whose columns are a multiple of 32, with their
    scales as (rows, columns / 32), are an 8-bit checkpoint that checkpoint8_read
    reads."""
    if bits == 32:
        return torch.zeros_like(param, dtype=torch.float32), torch.zeros_like(param, dtype=torch.float32)
    if bits != 8:
        raise ValueError("bits must be 8 or 32")
    one = lambda: (torch.zeros(param.shape, dtype=torch.uint8, device=param.device),  # noqa: E731
                   torch.zeros(-(-param.numel() // E4M3_BLOCK), dtype=torch.uint8, device=param.device))
    return one(), one()


def _few(t, name, dtype, n, dev):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.numel() == n and t.is_contiguous()
            and t.get_device() == dev):
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor of {n} on the same device")
    return t.data_ptr()


def adamw(tensors, step, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
          factors=None, seed: int = 0):
    """One step of AdamW over `tensors` (an AdamWTensors) on the current stream.

    step: its number, 1 the first: an int, or an int64 device tensor of one element
    for calls that are captured (below 1: nothing is changed).  factors: a float32
    device tensor of two, what lr and every gradient are multiplied by.  eps: 0, or
    1e-30 to 1e30.  seed: of the random rounding of 8-bit moments (mod 2^64)."""
    if not isinstance(tensors, AdamWTensors):
        raise TypeError("tensors must be an AdamWTensors (adamw_tensors)")
    dev = tensors.device
    if dev is None:
        return
    at = None
    if isinstance(step, torch.Tensor):
        at, step = _few(step, "step", torch.int64, 1, dev), 0
    f = _few(factors, "factors", torch.float32, 2, dev) if factors is not None else None
    _call(lib.hg_adamw, "hg_adamw", dev, tensors.count, tensors.array, int(step), at, lr, betas[0], betas[1], eps,
          weight_decay, f, seed & 0xffffffffffffffff)
