"""Python binding of include/hgemm_logprobs.h: log probabilities of given tokens,
entropy and the most probable tokens of rows of logits, and their gradient.
Argument marshalling only; re-exported by the package.

Logits are a matrix as in layer.py, float16, bfloat16 or float32; everything that
a row has one of is a contiguous vector.
"""
import ctypes

import torch

from . import HG_BF16, HG_F16, HG_F32, lib
from .adapters import _index
from .layer import _ONLY, _call, _device, _i64, _int, _matrix, _mp, _new_room, _room, _size, _vector, _vp

EXPORTS_LOGPROBS = ("hg_logprobs", "hg_logprobs_workspace_size", "hg_logprobs_grad")
_LOGITS = {torch.float16: HG_F16, torch.bfloat16: HG_BF16, torch.float32: HG_F32}
_float = ctypes.c_float

lib.hg_logprobs.argtypes = [_i64, _i64, _mp, _float, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _i64, _vp]
lib.hg_logprobs.restype = _int
lib.hg_logprobs_workspace_size.argtypes = [_i64, _i64, _int]
lib.hg_logprobs_workspace_size.restype = _i64
lib.hg_logprobs_grad.argtypes = [_i64, _i64, _mp, _float, _vp, _vp, _vp, _vp, _vp, _mp, _vp]
lib.hg_logprobs_grad.restype = _int


def _dense(t, name, shape, dtype, dev):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev):
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor of shape {shape} on the same device")
    return t.data_ptr()


def logprobs_workspace_size(X, top: int = 0) -> int:
    """Bytes of workspace logprobs needs for these logits and so many of the most probable tokens
    (hg_logprobs_workspace_size)."""
    dev = _device(X, "X")
    _, (M, V) = _matrix(X, "X", _LOGITS, dev)
    return _size(lib.hg_logprobs_workspace_size, "hg_logprobs_workspace_size", dev, M, V, int(top))


def logprobs_workspace(X, top: int = 0):
    """A workspace for logprobs calls on such logits (None if they need none)."""
    return _new_room(logprobs_workspace_size(X, top), X)


def logprobs(X, tokens=None, logp=None, entropy=None, stats=None, top=None, scale: float = 1.0, work=None):
    """What rows of logits X (M, V) stand for, with p = softmax(scale·X), on the
    current stream: writes those of the outputs that are given and returns
    (logp, entropy, stats, top).

    tokens (M,) int64: logp (M,) float32 gets log p of each row's token, 0 where
    it is outside 0 .. V-1 (no token).  entropy (M,) float32.  stats (M, 2)
    float32: for logprobs_grad.  top: a pair of (M, k) tensors, int64 numbers of
    the k <= 32 most probable tokens (equal ones: the lower number first) and
    float32 log probabilities, or None in place of either.  `work`: device tensor
    of at least logprobs_workspace_size(X, k) bytes (allocated with torch when
    None and needed)."""
    dev = _device(X, "X")
    x, (M, V) = _matrix(X, "X", _LOGITS, dev)
    t = l = e = st = ids = tl = wptr = None
    k = wbytes = 0
    if tokens is not None:
        t = _index(tokens, "tokens", M, dev)
    if logp is not None:
        if tokens is None:
            raise ValueError("logp needs tokens")
        l = _vector(logp, "logp", M, dev)
    if entropy is not None:
        e = _vector(entropy, "entropy", M, dev)
    if stats is not None:
        st = _dense(stats, "stats", (M, 2), torch.float32, dev)
    if top is not None:
        if not (isinstance(top, (tuple, list)) and len(top) == 2):
            raise TypeError("top must be a pair (numbers, log probabilities)")
        given = [v for v in top if v is not None]
        if not given or not isinstance(given[0], torch.Tensor) or given[0].dim() != 2:
            raise TypeError("top must be a pair of 2-D tensors, one of which may be None")
        k = given[0].shape[1]
        if top[0] is not None:
            ids = _dense(top[0], "top's numbers", (M, k), torch.int64, dev)
        if top[1] is not None:
            tl = _dense(top[1], "top's log probabilities", (M, k), torch.float32, dev)
    if work is None:
        work = _new_room(_size(lib.hg_logprobs_workspace_size, "hg_logprobs_workspace_size", dev, M, V, k), X)
    if work is not None:
        wptr, wbytes = _room(work, dev)
    _call(lib.hg_logprobs, "hg_logprobs", dev, M, V, x, scale, t, l, e, st, k, ids, tl, wptr, wbytes)
    return logp, entropy, stats, top


def logprobs_grad(X, tokens, stats, dX, dlogp=None, dentropy=None, entropy=None, scale: float = 1.0):
    """The gradient of logprobs on the current stream: dX = scale·(dlogp·(1[token]
    - p) - dentropy·p·(log p + entropy)); returns dX.

    X, tokens, stats, entropy and scale as logprobs took or gave them (entropy is
    needed only for dentropy), dlogp and dentropy (M,) float32, None being 0, dX
    (M, V) of X's type or X itself (in place)."""
    dev = _device(X, "X")
    x, (M, V) = _matrix(X, "X", _LOGITS, dev)
    d, shape = _matrix(dX, "dX", _ONLY[X.dtype], dev)
    if shape[0] != M or shape[1] != V:
        raise ValueError(f"dX {tuple(shape)} does not match X {(M, V)}")
    st = _dense(stats, "stats", (M, 2), torch.float32, dev)
    t = e = l = h = None
    if tokens is not None:
        t = _index(tokens, "tokens", M, dev)
    if dlogp is not None:
        if tokens is None:
            raise ValueError("dlogp needs tokens")
        l = _vector(dlogp, "dlogp", M, dev)
    if dentropy is not None:
        if entropy is None:
            raise ValueError("dentropy needs entropy")
        h = _vector(dentropy, "dentropy", M, dev)
        e = _vector(entropy, "entropy", M, dev)
    _call(lib.hg_logprobs_grad, "hg_logprobs_grad", dev, M, V, x, scale, t, st, e, l, h, d)
    return dX
