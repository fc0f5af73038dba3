"""Argument checks of include/hgemm_adamw.h and of its Python binding (CPU only, as
test_linear_abi.py; pointers are fake addresses)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, F32, BF16, E4M3 = 0, 1, 2, 3
P = [0x10000000 * (i + 1) for i in range(16)]        # addresses 256 MiB apart
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def api(hg):
    import half_precision_gemm_amd.optimizer as optimizer
    return optimizer


def tensor(api, **kw):
    d = dict(param=P[0], master=None, grad=P[1], m=P[2], m_scales=P[3], v=P[4], v_scales=P[5], n=100, param_type=BF16,
             grad_type=BF16, state_type=E4M3)
    return api.AdamWTensor(**{**d, **kw})


def step(api, tensors=None, count=None, t=1, dt=None, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, decay=0.1, factors=None):
    tensors = [tensor(api, n=0)] if tensors is None else tensors
    array = (api.AdamWTensor * max(1, len(tensors)))(*tensors) if tensors is not False else None
    return api.lib.hg_adamw(len(tensors) if count is None else count, array, t, dt, lr, b1, b2, eps, decay, factors, 0, None)


def test_header_and_exports_agree(api, hg):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "hgemm_adamw.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert names == set(hg.EXPORTS_ADAMW)
    so = ctypes.CDLL(hg.LIB_PATH)
    assert all(hasattr(so, n) for n in names)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), -1), (dict(count=(1 << 20) + 1), -1), (dict(tensors=False, count=1), -2), (dict(t=0), -3), (dict(t=-5), -3),
    (dict(dt=P[9] + 4), -4), (dict(lr=-1.0), -5), (dict(lr=NAN), -5), (dict(lr=INF), -5), (dict(lr=1e39), -5),
    (dict(b1=1.0), -6), (dict(b1=-0.1), -6), (dict(b1=NAN), -6), (dict(b2=1.0), -7), (dict(b2=NAN), -7), (dict(eps=-1.0), -8),
    (dict(eps=INF), -8), (dict(eps=9e-31), -8), (dict(eps=1.1e30), -8), (dict(eps=NAN), -8), (dict(decay=-1.0), -9), (dict(decay=NAN), -9), (dict(factors=P[9] + 2), -10),
    (dict(count=-1, t=0), -1), (dict(), 0), (dict(t=0, dt=P[9]), 0), (dict(tensors=[]), 0),
])
def test_refusals(api, kw, code):
    assert step(api, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=(1 << 36) + 1), dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(m_scales=None),
    dict(v_scales=None), dict(param=P[0] + 1), dict(grad=P[1] + 1), dict(grad_type=F32, grad=P[1] + 2),
    dict(state_type=F32, m=P[2] + 2), dict(state_type=F32, v=P[4] + 2), dict(master=P[6] + 2), dict(param_type=E4M3),
    dict(grad_type=E4M3), dict(state_type=BF16), dict(param_type=F32, master=P[6]), dict(param_type=7),
    dict(grad=P[0] + 198), dict(m=P[0]), dict(v=P[2] + 99), dict(m_scales=P[2] + 50), dict(v_scales=P[3] + 3),
    dict(master=P[1] - 398), dict(v=P[1]),
])
def test_bad_tensors(api, kw):
    good, bad = tensor(api, n=0), tensor(api, **kw)
    assert step(api, [good, bad], t=0) == -2 and step(api, [bad], t=0) == -2
    assert api.lib.hg_adamw_check(1, ctypes.byref(bad)) == -2


def test_arrays_on_the_step_or_the_factors(api):
    t = tensor(api)
    assert step(api, [t], dt=P[0] + 192) == -4 and step(api, [t], factors=P[4] + 96) == -10
    assert step(api, [t], t=0, factors=P[4] + 104) == -3


def test_overlaps_across_tensors(api):
    def check(*tensors):
        array = (api.AdamWTensor * len(tensors))(*tensors)
        return api.lib.hg_adamw_check(len(tensors), array)

    apart = lambda by, **kw: tensor(api, **{**{k: P[i] + by for i, k in enumerate(  # noqa: E731
        ("param", "grad", "m", "m_scales", "v", "v_scales"))}, **kw})
    first = apart(0)
    assert check(first) == 0 and check(first, apart(200)) == 0 and check(apart(200), first, apart(400)) == 0
    assert check(first, apart(200, grad=P[1])) == 0                       # gradients may be shared
    assert check(first, first) == -2                                      # the same tensor twice
    assert check(first, apart(200, param=P[0] + 198)) == -2 and check(first, apart(200, m=P[2] + 99)) == -2
    assert check(first, apart(200, v_scales=P[5] + 3)) == -2 and check(first, apart(200, v_scales=P[5] + 4)) == 0
    assert check(first, apart(200, grad=P[0])) == -2 and check(first, apart(200, m=P[1])) == -2
    assert check(first, apart(200, n=0, param=P[0])) == 0                 # has no elements
    many = [apart(200 * i) for i in range(300)]
    assert check(*many) == 0 and check(*many, apart(60000, v=P[4] + 200 * 150)) == -2


def test_binding_refuses_before_the_library(hg):
    p = torch.zeros(40)
    m, v = hg.adamw_state(p)
    with pytest.raises(ValueError, match="device tensor"):
        hg.adamw_tensors([p], [p], [m], [v])
    with pytest.raises(ValueError, match="one length"):
        hg.adamw_tensors([p], [], [m], [v])
    with pytest.raises(TypeError, match="torch.Tensor"):
        hg.adamw_tensors([1], [p], [m], [v])
    with pytest.raises(TypeError, match="AdamWTensors"):
        hg.adamw([p], 1)
    with pytest.raises(ValueError, match="bits"):
        hg.adamw_state(p, 16)
    hg.adamw(hg.adamw_tensors([], [], [], []), 1)
    m8, v8 = hg.adamw_state(torch.zeros(3, 33), 8)
    assert m8[0].shape == (3, 33) and m8[1].shape == (4,) and v8[0].dtype == v8[1].dtype == torch.uint8


def test_forms_of_a_moment(api):
    f = api._moment
    x = torch.zeros(33)
    assert f(x, "m", 33, -1)[1:] == (None, F32)
    assert f((torch.zeros(33).byte(), torch.zeros(2).byte()), "m", 33, -1)[2] == E4M3
    for bad, what in ((x[:32], "elements"), (x[::2], "contiguous"), ((torch.zeros(33).byte(), torch.zeros(1).byte()), "elements")):
        with pytest.raises(ValueError, match=what):
            f(bad, "m", 33, -1)
    for bad, what in ((x.half(), "dtype"), ((x, x), "dtype"), ([x], "pair"), ((x.byte(), 3), "torch.Tensor")):
        with pytest.raises(TypeError, match=what):
            f(bad, "m", 33, -1)
    with pytest.raises(ValueError, match="one device"):
        f(x, "m", 33, 0)
