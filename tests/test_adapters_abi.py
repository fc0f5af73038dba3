"""Argument checks of include/hgemm_adapters.h and of its Python binding (CPU
only, as test_linear_abi.py; pointers are fake addresses)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, F32, BF16, E4M3 = 0, 1, 2, 3
P = [0x10000000 * (i + 1) for i in range(12)]        # addresses 256 MiB apart
BIG = 1 << 20


@pytest.fixture(scope="module")
def api(hg):
    import half_precision_gemm_amd.adapters as adapters
    import half_precision_gemm_amd.layer as layer
    adapters.Matrix = layer.Matrix
    return adapters


def adapters_of(api, **kw):
    d = dict(which=P[7], scales=None, A=P[8], lda=16, stride_a=64, B=P[9], ldb=4, stride_b=32, count=3, rank=4, type=F16)
    return api.Adapters(**{**d, **kw})


def call(api, act=0, M=4, N=8, K=16, X=None, W=None, bias=P[2], R=None, Y=None, Z=None, ad=None, work=P[6],
         work_bytes=BIG):
    m = lambda v, d: api.Matrix(*(v or d)[:2], None, 0, (v or d)[2] if len(v or d) > 2 else F16)  # noqa: E731
    ad = None if ad is False else adapters_of(api, **(ad or {}))
    return api.lib.hg_linear_adapters(act, M, N, K, m(X, (P[0], 16)), m(W, (P[1], 16)), bias, R and m(R, None),
                                      m(Y, (P[4], 8)), Z and m(Z, None), ad, work, work_bytes, None)


def test_header_and_exports_agree(api, hg):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hgemm_adapters.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(hg.EXPORTS_ADAPTERS)
    so = ctypes.CDLL(hg.LIB_PATH)
    assert all(hasattr(so, n) for n in names)


@pytest.mark.parametrize("kw,code", [
    (dict(act=5), -1), (dict(M=-1), -2), (dict(N=BIG + 1), -3), (dict(K=-1), -4), (dict(X=(P[0], 15)), -5),
    (dict(W=(P[1], 16, BF16)), -6), (dict(bias=P[2] + 2), -7), (dict(R=(P[3], 7)), -8), (dict(Y=(P[4], 7)), -9),
    (dict(Z=(P[5], 8, F32)), -10), (dict(ad=False), -11), (dict(ad=dict(count=-1)), -11),
    (dict(ad=dict(count=BIG + 1)), -11), (dict(ad=dict(rank=-1)), -11), (dict(ad=dict(rank=257, ldb=257)), -11),
    (dict(ad=dict(type=BF16)), -11), (dict(ad=dict(lda=15)), -11), (dict(ad=dict(ldb=3)), -11),
    (dict(ad=dict(lda=(1 << 30) + 1)), -11), (dict(ad=dict(stride_a=-1)), -11),
    (dict(ad=dict(stride_b=(1 << 40) + 1)), -11), (dict(ad=dict(A=None)), -11), (dict(ad=dict(B=None)), -11),
    (dict(ad=dict(A=P[8] + 1)), -11), (dict(ad=dict(which=None)), -11), (dict(ad=dict(which=P[7] + 4)), -11),
    (dict(ad=dict(scales=P[7] + 2)), -11), (dict(Y=(P[0], 8)), -9), (dict(Z=(P[4] + 8, 8)), -10),
    # Y (64 bytes at P[4]) or Z on the adapters' arrays
    (dict(ad=dict(which=P[4] + 8)), -11), (dict(ad=dict(scales=P[4] + 60)), -11), (dict(ad=dict(A=P[4] - 64)), -11),
    (dict(ad=dict(B=P[4] - 64 * 2 - 30)), -11), (dict(Z=(P[9] + 2, 8)), -11),
    (dict(work=None), -12), (dict(work=P[6] + 8), -12), (dict(work=P[8] - 64), -12), (dict(work=P[4]), -12),
    (dict(work_bytes=255), -13), (dict(act=9, ad=False), -1),
])
def test_refusals(api, kw, code):
    assert call(api, **kw) == code


def test_what_is_not_read_is_not_checked(api):
    """Nothing to compute, or no adapters: their arrays may be missing."""
    none = dict(which=None, A=None, B=None)
    assert call(api, M=0, ad=none) == 0 and call(api, N=0, ad=none) == 0
    # (as hg_linear from here on: the first thing it does not get is the workspace)
    for ad in (dict(none, count=0), dict(none, rank=0)):
        assert call(api, M=100, K=8200, X=(P[0], 8200), W=(P[1], 8200), ad=ad, work=None) == -12


def test_binding_refuses_before_the_library(hg):
    x, w, y = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, 8)
    x, w, y = (v.half() for v in (x, w, y))
    with pytest.raises(ValueError, match="device tensor"):
        hg.linear_adapters(x, w, y, torch.zeros(4).long(), x[None], w[None])


def test_stacks(api):
    f = api._stack
    x = torch.zeros(3, 4, 16, dtype=torch.float16)
    assert f(x, "A", torch.float16, -1)[1:] == (16, 64, (3, 4, 16))
    assert f(x[:1, :1, :9], "A", torch.float16, -1)[1:] == (9, 0, (1, 1, 9))
    assert f(x[::2, ::2, 3:8], "A", torch.float16, -1)[1:] == (32, 128, (2, 2, 5))
    assert f(x[:1].expand(5, 4, 16), "A", torch.float16, -1)[1:] == (16, 0, (5, 4, 16))
    assert f(x[:, :0], "A", torch.float16, -1)[3] == (3, 0, 16)
    for bad, what in ((x[..., ::2], "unit stride"), (x[0], "3-D"), (x[:, :1].expand(3, 4, 16), "overlap")):
        with pytest.raises(ValueError, match=what):
            f(bad, "A", torch.float16, -1)
    with pytest.raises(TypeError, match="dtype"):
        f(x.float(), "A", torch.float16, -1)
    with pytest.raises(TypeError, match="torch.Tensor"):
        f([1], "A", torch.float16, -1)
    with pytest.raises(ValueError, match="one device"):
        f(x, "A", torch.float16, 0)
    assert api._index(torch.zeros(4).long(), "which", 4, -1)
    for bad in (torch.zeros(4), torch.zeros(3).long(), torch.zeros(8).long()[::2], torch.zeros(4, 1).long()):
        with pytest.raises(ValueError, match="int64 vector"):
            api._index(bad, "which", 4, -1)
