"""Which kernels the linear layer's calls take and how their products are cut
(CPU only: the host side of the library, compiled with launches that are only
written down; pointers are fake addresses that are never dereferenced)."""
import ctypes
import os
import subprocess

import pytest

import half_precision_gemm_amd.layer as layer

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
F16, F32, BF16, E4M3 = 0, 1, 2, 3
SPACE = 1 << 44                                    # between the fake matrices


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "half_precision_gemm_amd", "csrc"),
                    os.path.join(HERE, "linear_plan_stub.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    for name in ("hg_linear", "hg_linear_workspace_size", "hg_linear_grad", "hg_linear_grad_workspace_size"):
        f, g = getattr(lib, name), getattr(layer.lib, name)
        f.argtypes, f.restype = g.argtypes, g.restype
    lib.plan_launches.restype = ctypes.c_char_p
    return lib


def mat(i, cols, type=BF16, ld=None):
    return layer.Matrix((i + 1) * SPACE, ld or cols, (i + 1) * SPACE + SPACE // 2, -(-cols // 32), type)


def launches(lib):
    out = []
    for line in lib.plan_launches().decode().splitlines():
        kernel, *rest = line.split()
        out.append((kernel, {k: int(v) for k, v in (r.split("=") for r in rest)}))
    return out


def linear(lib, M, N, K, out=BF16, save=None, work_bytes=None, ldx=None, ldw=None):
    X, W, Y, Z = mat(0, K, ld=ldx), mat(1, K, ld=ldw), mat(2, N, out), mat(3, N, save) if save is not None else None
    if work_bytes is None:
        work_bytes = lib.hg_linear_workspace_size(M, N, K, X, W)
    st = lib.hg_linear(4, M, N, K, X, W, None, None, Y, Z, 9 * SPACE, work_bytes, None)
    return st, launches(lib)


def grad(lib, M, N, K, x=BF16, z=BF16, want="xwb"):
    dY, W, X, Z = mat(0, N), mat(1, K), mat(2, K, x), mat(3, N, z)
    work = lib.hg_linear_grad_workspace_size(M, N, K, dY, W, X)
    st = lib.hg_linear_grad(4, M, N, K, dY, W, X, Z, mat(4, K) if "x" in want else None,
                            mat(5, K, F32) if "w" in want else None, 7 * SPACE if "b" in want else None, 0, 9 * SPACE,
                            work, None)
    return st, launches(lib)


MOST = 0xffffffff // 256                           # workgroups of 256 threads: HIP refuses a launch of 2^32 threads


@pytest.mark.parametrize("M,N,K", [(1 << 30, 16, 16), (1 << 30, 16, 7), (1 << 30, 8, 8), ((1 << 30) - 64, 64, 8),
                                   ((1 << 29) + 1, 65, 8), (1 << 29, 128, 24), (1 << 30, 129, 1), (1 << 20, 1 << 20, 64),
                                   (1 << 25, 4096, 64)])
def test_launches_of_the_tallest_products(lib, M, N, K):
    """Every launch stays below 2^32 threads at any size that is allowed."""
    st, done = linear(lib, M, N, K)
    assert st == 0 and done and all(d["blocks"] <= MOST for _, d in done), done


@pytest.mark.parametrize("want", ["xwb", "xb", "wb", "x", "w"])
@pytest.mark.parametrize("M,N,K", [(1 << 30, 16, 16), (1 << 30, 8, 64), (1 << 30, 64, 8), ((1 << 29) + 1, 8, 65),
                                   (1 << 30, 1, 129), (1 << 30, 200, 200), (64, 1 << 20, 1 << 20), (1 << 20, 1 << 20, 64)])
def test_launches_of_the_tallest_gradients(lib, M, N, K, want):
    st, done = grad(lib, M, N, K, want=want)
    assert st == 0 and done and all(d["blocks"] <= MOST for _, d in done), done


# M, N, K, whether row by row with Z in 16 bits and in 8 bits.  8 bits: 32 rows of W in a workgroup at any N, so half
# as many workgroups; the measured figures stand beside the choice.
FEW = [(16, 4096, 4096, True, True), (64, 4096, 4096, True, False), (1, 2048, 8192, True, False),
       (16, 2048, 8192, True, False), (32, 4096, 8192, True, False), (64, 2048, 4096, True, False),
       (16, 1024, 1024, True, True), (64, 4096, 1024, True, False), (16, 8192, 2048, True, True),
       (16, 16384, 4096, True, True), (16, 4096, 4098, True, False), (65, 4096, 4096, False, False)]


@pytest.mark.parametrize("M,N,K,rows16,rows8", FEW)
def test_few_rows_are_priced_as_they_are_launched(lib, M, N, K, rows16, rows8):
    for save, rows in ((None, rows16), (BF16, rows16), (E4M3, rows8)):
        st, done = linear(lib, M, N, K, save=save)
        assert st == 0 and ("rowwise" in [k for k, _ in done]) == rows, (save, done)


@pytest.mark.parametrize("M", [1, 7, 16, 33, 64, 100])
@pytest.mark.parametrize("N,K,ldx,ldw", [(2048, 8192, None, None), (4096, 4096, None, None), (4096, 4098, None, None),
                                         (1000, 8191, 8192, 8193), (512, 16384, 16386, None), (64, 100, None, 101)])
def test_one_workspace_for_any_saved_form(lib, M, N, K, ldx, ldw):
    """hg_linear_workspace_size does not see Z: its size is enough for every form of it."""
    for save in (None, BF16, E4M3):
        assert linear(lib, M, N, K, save=save, ldx=ldx, ldw=ldw)[0] == 0, save
