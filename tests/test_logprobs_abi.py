"""Argument checks of include/hgemm_logprobs.h and of its Python binding (CPU
only, as test_linear_abi.py; pointers are fake addresses)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, F32, BF16, E4M3 = 0, 1, 2, 3
P = [0x10000000 * (i + 1) for i in range(12)]        # addresses 256 MiB apart
NULL = object()
INF = float("inf")


@pytest.fixture(scope="module")
def api(hg):
    import half_precision_gemm_amd.layer as layer
    import half_precision_gemm_amd.logits as logits
    logits.Matrix = layer.Matrix
    return logits


def mat(api, data, ld, type=BF16):
    return api.Matrix(data, ld, None, 0, type)


def forward(api, M=4, V=100, X=None, scale=1.0, tokens=P[1], logp=P[2], entropy=P[3], stats=P[4], top=5, ids=P[5], tl=P[6],
            work=P[7], work_bytes=1 << 20):
    X = None if X is NULL else mat(api, *(X or (P[0], 100)))
    return api.lib.hg_logprobs(M, V, X, scale, tokens, logp, entropy, stats, top, ids, tl, work, work_bytes, None)


def backward(api, M=4, V=100, X=None, scale=1.0, tokens=P[1], stats=P[2], entropy=P[3], dl=P[4], dh=P[5], dX=None):
    X, dX = (None if m is NULL else mat(api, *(m or (p, 100))) for m, p in ((X, P[0]), (dX, P[6])))
    return api.lib.hg_logprobs_grad(M, V, X, scale, tokens, stats, entropy, dl, dh, dX, None)


def test_header_and_exports_agree(api, hg):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hgemm_logprobs.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(hg.EXPORTS_LOGPROBS)
    so = ctypes.CDLL(hg.LIB_PATH)
    assert all(hasattr(so, n) for n in names)


LONG = dict(V=40000, X=(P[0], 40000))                # several parts: a workspace is needed


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(M=(1 << 30) + 1), -1), (dict(V=0), -2), (dict(V=(1 << 20) + 1), -2), (dict(X=NULL), -3),
    (dict(X=(P[0], 99)), -3), (dict(X=(P[0], 100, E4M3)), -3), (dict(X=(P[0] + 1, 100)), -3),
    (dict(X=(P[0] + 2, 100, F32)), -3), (dict(X=(None, 100)), -3), (dict(scale=0.0), -4), (dict(scale=-1.0), -4),
    (dict(scale=INF), -4), (dict(scale=float("nan")), -4), (dict(scale=1.1e30), -4), (dict(tokens=None), -5), (dict(tokens=P[1] + 4), -5),
    (dict(logp=P[2] + 2), -6), (dict(entropy=P[3] + 1), -7), (dict(stats=P[4] + 2), -8), (dict(top=-1), -9),
    (dict(top=33), -9), (dict(top=5, V=4), -9), (dict(ids=P[5] + 4), -10), (dict(tl=P[6] + 2), -11),
    (dict(logp=P[0] + 4), -6), (dict(logp=P[1]), -6), (dict(entropy=P[2] + 12), -7), (dict(stats=P[3] + 8), -8),
    (dict(ids=P[4] + 24), -10), (dict(tl=P[5] + 8), -11), (dict(tl=P[0]), -11),
    (dict(LONG, work=None), -12), (dict(LONG, work=P[7] + 8), -12), (dict(LONG, work=P[0]), -12),
    (dict(LONG, work=P[6]), -12), (dict(LONG, work_bytes=64), -13), (dict(M=-1, V=0, scale=0.0), -1),
])
def test_forward_refusals(api, kw, code):
    assert forward(api, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(V=0), -2), (dict(X=NULL), -3), (dict(X=(P[0], 99)), -3), (dict(scale=0.0), -4),
    (dict(tokens=None), -5), (dict(tokens=P[1] + 4), -5), (dict(stats=None), -6), (dict(stats=P[2] + 2), -6),
    (dict(entropy=None), -7), (dict(entropy=P[3] + 2), -7), (dict(dl=P[4] + 1), -8), (dict(dh=P[5] + 2), -9),
    (dict(dX=NULL), -10), (dict(dX=(P[6], 99)), -10), (dict(dX=(P[6], 100, F32)), -10), (dict(dX=(P[6], 100, F16)), -10),
    (dict(dX=(P[0] + 2, 100)), -10), (dict(dX=(P[0], 101)), -10), (dict(dX=(P[1], 100)), -10), (dict(dX=(P[2] - 64, 100)), -10),
    (dict(dX=(P[3], 100)), -10), (dict(dX=(P[4], 100)), -10), (dict(dX=(P[5], 100)), -10),
])
def test_gradient_refusals(api, kw, code):
    assert backward(api, **kw) == code


def test_empty_calls_touch_nothing(api):
    none = dict(tokens=None, stats=None, entropy=None)
    assert forward(api, M=0, X=(None, 100), logp=None, ids=None, tl=None, work=None, work_bytes=0, **none) == 0
    assert backward(api, M=0, X=(None, 100), dX=(None, 100), dl=None, dh=None, **none) == 0


def test_workspace_sizes(api):
    size = api.lib.hg_logprobs_workspace_size
    assert size(-1, 8, 0) == -1 and size(8, 0, 0) == -2 and size(8, 8, 9) == -3 and size(8, 8, -1) == -3
    assert size(0, 100, 4) == 0 and size(5, 2000, 32) == 0
    for M in (1, 100, 5000):
        for V in (2049, 50264, 1 << 20):
            a, b = size(M, V, 0), size(M, V, 32)
            assert 0 <= a <= b <= M * 65 * (16 + 32 * 8) + 512


def test_binding_refuses_before_the_library(api, hg):
    x = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        hg.logprobs(x)
    with pytest.raises(TypeError, match="torch.Tensor"):
        hg.logprobs([1])
    with pytest.raises(TypeError, match="dtype"):
        hg.logprobs_grad(x.double(), None, x, x)
    with pytest.raises(ValueError, match="stats must be a contiguous float32"):
        api._dense(torch.zeros(4, 3), "stats", (4, 2), torch.float32, -1)
    assert api._dense(torch.zeros(4, 2), "stats", (4, 2), torch.float32, -1)
