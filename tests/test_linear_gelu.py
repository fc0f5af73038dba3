"""The error that the linear layer's GELU states for its polynomial of the
normal distribution's tail (CPU only: the coefficients are read from the
source and evaluated in fp32)."""
import math
import os
import re

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def coefficients():
    src = open(os.path.join(ROOT, "half_precision_gemm_amd", "csrc", "hg_linear.h")).read()
    body = src[src.index("float log2_tail(float x)"):]
    body = body[:body.index("\n}")]
    return [np.float32(c) for c in re.findall(r"-?\d\.\d+(?:e-?\d+)?(?=f[;)])", body)]


def tail32(x):
    """2^polynomial in fp32: fused multiply-adds (the product is exact in 64 bits), the power rounded once."""
    c = coefficients()
    assert len(c) == 9
    q = np.full_like(x, c[0])
    for v in c[1:]:
        with np.errstate(over="ignore"):                   # far out it falls to -inf
            q = (q.astype(np.float64) * x + np.float64(v)).astype(np.float32)
    return np.exp2(q.astype(np.float64)).astype(np.float32).astype(np.float64)


def exact(x):
    return torch.special.erfc(torch.from_numpy(x.astype(np.float64)) / math.sqrt(2)).numpy() / 2


def test_absolute_error():
    """Of 1 - Phi, everywhere."""
    x = np.concatenate([np.linspace(0, 14, 2000001), np.geomspace(1e-30, 3e38, 200001)]).astype(np.float32)
    got = tail32(x)
    assert np.isfinite(got).all() and (got >= 0).all()
    assert np.abs(got - exact(x)).max() <= 7.3e-8


def test_relative_error():
    """2e-5 of the tail up to 3, 3.1e-4 up to 5.6."""
    x = np.linspace(0, 5.6, 2000001).astype(np.float32)
    rel = np.abs(tail32(x) / exact(x) - 1)
    assert rel[x <= 3].max() <= 2.0e-5 and rel.max() <= 3.1e-4, (rel[x <= 3].max(), rel.max())
