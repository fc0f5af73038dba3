"""Argument checks of include/hgemm_linear.h and of its Python binding (CPU
only; every call returns before the library touches the HIP runtime; pointers
are fake addresses that are never dereferenced)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, F32, BF16, E4M3 = 0, 1, 2, 3
P = [0x10000000 * (i + 1) for i in range(12)]        # addresses 256 MiB apart
NULL = object()


@pytest.fixture(scope="module")
def api(hg):
    import half_precision_gemm_amd.layer as layer
    return layer


def mat(api, data, ld, type=F16, scales=None, lds=0):
    return api.Matrix(data, ld, scales, lds, type)


def linear(api, act=0, M=4, N=8, K=16, X=None, W=None, bias=P[2], R=None, Y=None, Z=None, work=P[6],
           work_bytes=1 << 20):
    pick = lambda v, d: None if v is NULL else (d if v is None else v)  # noqa: E731
    return api.lib.hg_linear(act, M, N, K, pick(X, mat(api, P[0], 16)), pick(W, mat(api, P[1], 16)), bias, R,
                             pick(Y, mat(api, P[4], 8)), Z, work, work_bytes, None)


def grad(api, act=4, M=4, N=8, K=16, dY=None, W=None, X=None, Z=None, dX=None, dW=None, db=P[7], acc=0, work=P[8],
         work_bytes=1 << 20):
    pick = lambda v, d: None if v is NULL else (d if v is None else v)  # noqa: E731
    return api.lib.hg_linear_grad(act, M, N, K, pick(dY, mat(api, P[0], 8)), pick(W, mat(api, P[1], 16)),
                                  pick(X, mat(api, P[2], 16)), pick(Z, mat(api, P[3], 8)),
                                  pick(dX, mat(api, P[5], 16)), pick(dW, mat(api, P[6], 16)), db, acc, work, work_bytes,
                                  None)


def test_header_and_exports_agree(api, hg):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hgemm_linear.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(hg.EXPORTS_LINEAR)
    so = ctypes.CDLL(hg.LIB_PATH)
    assert all(hasattr(so, n) for n in names)
    assert (hg.ACT_NONE, hg.ACT_RELU, hg.ACT_GELU, hg.ACT_GELU_TANH, hg.ACT_SILU) == (0, 1, 2, 3, 4)


BIG = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(act=-1), -1), (dict(act=5), -1), (dict(M=-1), -2), (dict(M=(1 << 30) + 1), -2), (dict(N=-1), -3),
    (dict(N=BIG + 1), -3), (dict(K=-1), -4), (dict(K=BIG + 1), -4), (dict(X=NULL), -5), (dict(W=NULL), -6),
    (dict(Y=NULL), -9), (dict(work=None, M=100, K=8200, X=(P[0], 8200), W=(P[1], 8200)), -11),
    (dict(work=P[6] + 8, M=100, K=8200, X=(P[0], 8200), W=(P[1], 8200)), -11),
    (dict(work_bytes=0, M=100, K=8200, X=(P[0], 8200), W=(P[1], 8200)), -12),
    (dict(X=(None, 16)), -5), (dict(X=(P[0] + 1, 16)), -5), (dict(X=(P[0], 15)), -5), (dict(X=(P[0], (1 << 30) + 1)), -5),
    (dict(X=(P[0], 16, F32)), -5), (dict(X=(P[0], 16, E4M3)), -5), (dict(W=(P[1], 16, BF16)), -6), (dict(W=(P[1], 8)), -6),
    (dict(bias=P[2] + 2), -7), (dict(R=(P[3], 7)), -8), (dict(R=(P[3], 8, F32)), -8), (dict(Y=(P[4], 7)), -9),
    (dict(Y=(P[4], 8, BF16)), -9), (dict(Y=(P[4], 8, E4M3)), -9), (dict(Y=(P[4] + 2, 8, F32)), -9),
    (dict(Z=(P[5], 8, F32)), -10), (dict(Z=(P[5], 8, E4M3)), -10), (dict(Z=(P[5], 8, E4M3, P[7], 0)), -10),
    (dict(Y=(P[0] + 16, 8)), -9), (dict(Y=(P[1], 8)), -9), (dict(Y=(P[2], 8)), -9), (dict(R=(P[4] + 16, 8)), -9),
    (dict(R=(P[4], 16)), -9), (dict(Z=(P[4] + 8, 8)), -10), (dict(Z=(P[0], 8)), -10),
    (dict(Z=(P[5], 8, E4M3, P[5] + 8, 1)), -10), (dict(Z=(P[5], 8, E4M3, P[4], 1)), -10),
    (dict(M=100, K=8200, X=(P[0], 8200), W=(P[1], 8200), work=P[4]), -11), (dict(M=100, K=8200, X=(P[0], 8200), W=(P[1], 8200), work=P[0]), -11),
])
def test_linear_refusals(api, kw, code):
    kw = {k: mat(api, *v[:2], *(v[2:3] or (F16,)), *v[3:]) if isinstance(v, tuple) else v for k, v in kw.items()}
    assert linear(api, **kw) == code


@pytest.mark.parametrize("X,Y,Z,code", [
    ((0, 8224), (16400, 8224), (16416, 8224), -11),       # X, Y and Z: bytes 0, 16400, 16416 of rows of 16448
    ((0, 8224), (16398, 8224), (16416, 8224), -9),        # Y on X's last column
    ((0, 8224), (16434, 8224), (16400, 8224), -9),        # Y's end on the next row's X
    ((0, 8224), (16400, 8224), (16414, 8224), -10),       # Z on Y's last column
    ((0, 8224), (16400, 8224), (16448 * 100, 8224), -11),       # behind X's last row
    ((0, 8224), (16400, 8224), (16448 * 99 + 18, 8224), -10),   # in it, on X
    ((0, 8224), (16400, 8225), (16416, 8224), -9),        # another pitch
])
def test_columns_of_one_array(api, X, Y, Z, code):
    """M = 100, N = 8, K = 8200 in 16 bits; what does not overlap goes on to the missing workspace."""
    X, Y, Z = (mat(api, P[0] + at, ld) for at, ld in (X, Y, Z))
    assert linear(api, M=100, K=8200, X=X, W=mat(api, P[1], 8200), Y=Y, Z=Z, work=None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(act=9), -1), (dict(M=-1), -2), (dict(N=BIG + 1), -3), (dict(K=-1), -4), (dict(dY=NULL), -5),
    (dict(dY=(P[0], 8, F32)), -5), (dict(dY=(P[0], 7)), -5), (dict(W=NULL), -6), (dict(W=(P[1], 15)), -6),
    (dict(W=(P[1], 16, BF16)), -6), (dict(X=NULL), -7), (dict(X=(P[2], 16, F32)), -7), (dict(X=(P[2], 16, E4M3)), -7),
    (dict(X=(P[2], 16, E4M3, P[9], 0)), -7), (dict(Z=NULL), -8), (dict(Z=(None, 8)), -8), (dict(Z=(P[3], 7)), -8),
    (dict(dX=(P[5], 16, F32)), -9), (dict(dX=(P[5], 15)), -9), (dict(dW=(P[6], 16, BF16)), -10),
    (dict(dW=(P[6] + 2, 16, F32)), -10), (dict(db=P[7] + 1), -11), (dict(acc=2), -12), (dict(work=None), -13),
    (dict(work=P[8] + 4), -13), (dict(work_bytes=16), -14), (dict(dX=(P[0], 16)), -9), (dict(dX=(P[3], 16)), -9),
    (dict(dW=(P[5] + 32, 16)), -10), (dict(dW=(P[2], 16)), -10), (dict(db=P[6]), -11), (dict(db=P[0]), -11),
    (dict(work=P[5]), -13), (dict(work=P[1]), -13),
])
def test_grad_refusals(api, kw, code):
    kw = {k: mat(api, *v[:2], *(v[2:3] or (F16,)), *v[3:]) if isinstance(v, tuple) else v for k, v in kw.items()}
    assert grad(api, **kw) == code


@pytest.mark.parametrize("M,N,x,c,code", [
    (-1, 8, (P[0], 8), (P[1], 8, E4M3, P[2], 1), -1), (4, BIG + 1, (P[0], 8), (P[1], 8, E4M3, P[2], 1), -2),
    (4, 8, (P[0], 7), (P[1], 8, E4M3, P[2], 1), -3), (4, 8, (P[0], 8, F32), (P[1], 8, E4M3, P[2], 1), -3),
    (4, 8, (P[0], 8), (P[1], 8), -4), (4, 8, (P[0], 8), (P[1], 8, E4M3, None, 1), -4),
    (4, 33, (P[0], 33), (P[1], 33, E4M3, P[2], 1), -4), (4, 8, (P[0], 8), (P[0] + 8, 8, E4M3, P[2], 1), -4),
    (4, 8, (P[0], 8), (P[1], 8, E4M3, P[0], 1), -4), (4, 8, (P[0], 8), (P[1], 8, E4M3, P[1], 1), -4),
])
def test_checkpoint_write_refusals(api, M, N, x, c, code):
    assert api.lib.hg_checkpoint8_write(M, N, mat(api, *x), mat(api, *c), None) == code


def test_checkpoint_read_refusals(api):
    good = mat(api, P[1], 8, E4M3, P[2], 1)
    read = api.lib.hg_checkpoint8_read
    assert read(4, 8, mat(api, P[1], 8), mat(api, P[0], 8), None) == -3
    assert read(4, 8, good, mat(api, P[0], 8, F32), None) == -4
    assert read(4, 8, good, mat(api, P[1], 8), None) == -4            # over the codes
    assert read(4, 8, good, mat(api, P[2], 8), None) == -4            # over the scales
    assert read(4, 8, None, mat(api, P[0], 8), None) == -3


def test_empty_calls_touch_nothing(api):
    none = mat(api, None, 16)
    for kw in (dict(M=0), dict(N=0)):
        assert linear(api, X=none, W=none, Y=none, bias=None, work=None, work_bytes=0, **kw) == 0
    assert grad(api, M=0, N=0, dY=none, W=none, X=none, Z=none, dX=none, dW=none, db=None) == 0
    assert api.lib.hg_checkpoint8_write(0, 8, none, mat(api, None, 8, E4M3, None, 1), None) == 0
    assert api.lib.hg_checkpoint8_read(4, 0, mat(api, None, 8, E4M3, None, 1), none, None) == 0


def test_workspace_sizes(api):
    size = api.lib.hg_linear_workspace_size
    x, w = mat(api, P[0], 4096), mat(api, P[1], 4096)
    assert size(0, 4096, 4096, x, w) == 0 and size(64, 64, 0, x, w) == 0
    odd = mat(api, P[0], 4095)
    need = size(4096, 4096, 4095, odd, mat(api, P[1], 4095))
    assert need >= 2 * 4096 * 4096 * 2                                 # both copied to rows of 4096
    assert size(4096, 4096, 4096, mat(api, P[0] + 2, 4096), w) >= 4096 * 4096 * 2
    assert size(-1, 8, 8, x, w) == -1 and size(8, -1, 8, x, w) == -2 and size(8, 8, -1, x, w) == -3
    assert size(8, 8, 8, None, w) == -4 and size(8, 8, 8, x, None) == -5
    assert size(8, 8, 8, mat(api, P[0], 7), w) == -4 and size(8, 8, 8, x, mat(api, P[1], 8, BF16)) == -5
    gsize = api.lib.hg_linear_grad_workspace_size
    dy = mat(api, P[2], 4096)
    assert gsize(128, 4096, 4096, dy, w, x) >= 128 * 4096 * 2
    assert gsize(128, 4096, 4096, dy, w, mat(api, P[0], 4096, E4M3, P[3], 128)) >= 2 * 128 * 4096 * 2
    assert gsize(128, 4096, 4096, dy, None, None) >= 128 * 4096 * 2
    assert gsize(8, 8, 8, None, w, x) == -4 and gsize(8, 8, 8, dy, mat(api, P[1], 7), x) == -5
    assert gsize(8, 8, 8, dy, w, mat(api, P[0], 8, F32)) == -6


def test_first_bad_argument_wins(api):
    assert linear(api, act=7, M=-1) == -1
    assert linear(api, X=NULL, Y=NULL) == -5


def test_binding_refuses_before_the_library(hg):
    x = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        hg.linear(x, x, x)
    with pytest.raises(TypeError, match="torch.Tensor"):
        hg.linear([1], x, x)
    with pytest.raises(TypeError, match="dtype"):
        hg.linear(x.double(), x, x)
    with pytest.raises(ValueError, match="2-D"):
        hg.checkpoint8_write(x[0], x, x)
    with pytest.raises(TypeError, match="dtype"):
        hg.linear_grad(x.int(), x, x)
    codes, scales = hg.checkpoint8_empty(5, 70, "cpu")
    assert codes.shape == (5, 70) and scales.shape == (5, 3)
