"""The linear layer, its gradient and 8-bit checkpoints in 64 bits, from their
definitions (torch on the CPU), and the error bounds the tests hold the
kernels to.

Bounds.  u32 = 2^-24; `half(t)` is half a step of a type relative to the value
(bf16 2^-8, fp16 2^-11, fp32 2^-24); an fp16 result below the normal range is
off by at most 2^-25.

  * A sum of K exact products, fp32, any order: |error| <= (K + 2)·u32·Σ|x·w|
    (the usual worst case, bias included as one more term).
  * act: the fp32 evaluation is z·p with p a probability.  logistic: exp of a
    rounded argument is off by |x|·2^-23 + 2^-22 relative, which moves p by at
    most p(1-p)·that <= 0.28·2^-23 + 2^-24, and the reciprocal adds 2^-23; the
    normal distribution function's formula has 0.75e-7 < 2^-23 absolute and a
    dozen roundings of terms below 1.  Together under 2^-20, so |act| is off by
    |z|·2^-20, and |act'| by 2^-19·(1 + |z|·(1 + z²)·min(1, density)), taken as
    2^-17 (|z|^3 times the density or logistic's slope stays below 2).
  * |act'| <= 1.13 and |act''| <= 1 for every activation here.
"""
import math

import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
U32 = 2.0 ** -24
BLOCK = 32


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}.get(dtype, 2.0 ** -150)


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, 0.0, z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def linear(X, W, bias=None, name="none", R=None):
    """(Y, Z, bound on |Y|'s fp32 error, bound on |Z|'s) before the last rounding."""
    X, W = X.double(), W.double()
    z = X @ W.t()
    mag = X.abs() @ W.abs().t()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ez = (X.shape[1] + 2) * U32 * mag
    y = act(z, name)
    ey = 1.13 * ez + (z.abs() + ez) * 2.0 ** -20
    if R is not None:
        y = y + R.double()
        ey = ey + U32 * (y.abs() + ey)
    return y, z, ey, ez


def check(out, ref, err, what):
    """|out - ref| <= err + the rounding to out's type, NaN and inf in the same places."""
    o, t = out.detach().cpu().double(), out.dtype
    assert o.shape == ref.shape, (what, o.shape, ref.shape)
    lim = err + half(t) * (ref.abs() + err) + tiny(t)
    bad = ~((o - ref).abs() <= lim)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {float(o[i])!r}, "
                             f"expected {float(ref[i])!r} within {float(lim[i])!r}")


def grads(dY, W, X, Z, name):
    """{name: (value, bound)} of dz, dX, dW, dbias; the bounds hold the rounding of dz to dY's type
    (the products' operand) but not the last one."""
    t = dY.dtype
    dy, w, x, z = dY.double(), W.double(), X.double(), Z.double()
    dz = dy * slope(z, name)
    e = torch.zeros_like(dz) if name == "none" else dy.abs() * 2.0 ** -17
    d = e + U32 * dz.abs()
    r = d if name == "none" else d + half(t) * (dz.abs() + d) + tiny(t)     # rounded for the products
    a, M, N = dz.abs() + r, dz.shape[0], dz.shape[1]
    return {"dX": (dz @ w, r @ w.abs() + (N + 2) * U32 * (a @ w.abs())),
            "dW": (dz.t() @ x, r.t() @ x.abs() + (M + 2) * U32 * (a.t() @ x.abs())),
            "dbias": (dz.sum(0), d.sum(0) + (M + 2) * U32 * a.sum(0))}


def codes8(X):
    """(codes as float8 values, scale bytes) of a 16-bit matrix, by the definition: the exponent is searched, the
    code is the nearest of all e4m3 values, the even one of two."""
    fp16 = X.dtype == torch.float16
    rows, cols = X.shape
    nb = -(-cols // BLOCK)
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    grid = torch.sort(table[torch.isfinite(table) & (table >= 0)]).values           # 0 .. 448, ascending codes
    grid = torch.unique(grid)
    vals = torch.zeros(rows, cols, dtype=torch.float64)
    scales = torch.zeros(rows, nb, dtype=torch.int64)
    x = X.double()
    for b in range(nb):
        blk = x[:, b * BLOCK:(b + 1) * BLOCK]
        fin = torch.isfinite(blk)
        amax = torch.where(fin, blk.abs(), 0.0).amax(1)
        lo, hi = (-15, 8) if fp16 else (-117, 127)
        e = torch.full((rows,), lo)
        for _ in range(hi - lo):
            e = torch.where((amax > 448 * torch.exp2(e.double())) & (e < hi), e + 1, e)
        top = torch.where(e == (8 if fp16 else 120), 240.0, 448.0)      # 256·2^e is past the type's range
        v = (blk.abs() * torch.exp2(-e.double())[:, None])
        v = torch.where(fin, torch.minimum(v, top[:, None]), 0.0)
        k = torch.searchsorted(grid, v.contiguous()).clamp(1, len(grid) - 1)          # grid[k-1] < v <= grid[k]
        below, above = grid[k - 1], grid[k]
        up = (above - v < v - below) | ((above - v == v - below) & (k % 2 == 0))      # code k is even
        q = torch.where(v <= 0, 0.0, torch.where(up, above, below)) * torch.where(blk < 0, -1.0, 1.0)
        vals[:, b * BLOCK:(b + 1) * BLOCK] = torch.where(fin, q * torch.exp2(e.double())[:, None], float("nan"))
        scales[:, b] = e + 127
    return vals, scales.to(torch.uint8)


def values8(codes, scales):
    """What the codes stand for, in 64 bits."""
    c = codes.cpu().view(torch.float8_e4m3fn).float().double()
    s = torch.exp2(scales.cpu().double() - 127).repeat_interleave(BLOCK, 1)[:, :c.shape[1]]
    return c * s
