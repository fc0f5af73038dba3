"""Which kernels the linear layer with adapters takes, and that its workspace is
enough for any call (CPU only, as test_linear_plan.py)."""
import ctypes
import os
import subprocess

import pytest

import half_precision_gemm_amd.adapters as adapters
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
                    os.path.join(HERE, "adapters_plan_stub.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    for name in ("hg_linear", "hg_linear_adapters", "hg_linear_adapters_workspace_size", "hg_linear_workspace_size"):
        f, g = getattr(lib, name), getattr(layer.lib, name)
        f.argtypes, f.restype = g.argtypes, g.restype
    lib.plan_launches.restype = ctypes.c_char_p
    return lib


def mat(i, cols, type=BF16, ld=None):
    return layer.Matrix((i + 1) * SPACE, ld or cols, (i + 1) * SPACE + SPACE // 2, -(-cols // 32), type)


def call(lib, M, N, K, rank=16, count=4, save=None, ldx=None, ldw=None, short=0):
    X, W, Y, Z = mat(0, K, ld=ldx), mat(1, K, ld=ldw), mat(2, N), mat(3, N, save) if save is not None else None
    L = adapters.Adapters(5 * SPACE, None, 6 * SPACE, K, rank * K, 7 * SPACE, max(1, rank), N * max(1, rank), count, rank,
                          BF16)
    work = lib.hg_linear_adapters_workspace_size(M, N, K, rank, X, W)
    st = lib.hg_linear_adapters(4, M, N, K, X, W, None, None, Y, Z, L, 9 * SPACE, work - short, None)
    lines = [line.split() for line in lib.plan_launches().decode().splitlines()]
    return st, [(k, {a: int(b) for a, b in (r.split("=") for r in rest)}) for k, *rest in lines]


@pytest.mark.parametrize("M,N,K,rank,kernels", [
    (1, 4096, 4096, 16, ["rowwise"]), (1, 4096, 4096, 17, ["shrink_wide", "rowwise"]), (2, 4096, 4096, 16, ["shrink_wide", "rowwise"]),
    (1, 16384, 4096, 16, ["shrink_wide", "rowwise"]), (1, 4096, 4092, 16, ["shrink_wide", "rowwise"]), (64, 4096, 4096, 9, ["shrink_wide", "rowwise"]),
    (16, 1000, 777, 5, ["shrink_wide", "rowwise"]), (65, 512, 512, 16, ["shrink", "ring"]),
    (64, 50264, 2048, 16, ["shrink", "ring"]), (333, 1111, 777, 9, ["shrink", "loose"]),
    (128, 1024, 8192, 16, ["shrink", "ring", "reduce"]), (8192, 4096, 4096, 16, ["shrink", "tile"]),
    (8192, 4096, 4096, 24, ["shrink", "tile"]), (8192, 4096, 4096, 17, ["shrink", "ring"]),
    (8192, 4096, 4095, 16, ["shrink", "prepare", "tile"]),
])
def test_kernels(lib, M, N, K, rank, kernels):
    st, done = call(lib, M, N, K, rank)
    assert st == 0 and [k for k, _ in done] == kernels, done
    # T: fp32 up to a whole eight, or high and low halves up to 32
    up = -(-rank // 8) * 8
    assert kernels[0] == "rowwise" or done[0][1]["edge"] == (up if kernels[0] == "shrink_wide" else -(-2 * up // 32) * 32)


def test_without_adapters_it_is_the_layer(lib):
    for kw in (dict(rank=0), dict(count=0)):
        st, done = call(lib, 100, 512, 512, **kw)
        assert st == 0 and [k for k, _ in done] == ["ring"], done


@pytest.mark.parametrize("M", [1, 7, 16, 33, 64, 100, 3000])
@pytest.mark.parametrize("rank", [1, 8, 9, 16, 17, 64, 100, 256])
@pytest.mark.parametrize("N,K,ldx,ldw", [(2048, 8192, None, None), (4096, 4098, None, None), (1000, 8191, 8192, 8193),
                                         (512, 16384, 16386, None), (64, 100, None, 101)])
def test_one_workspace_for_any_saved_form(lib, M, rank, N, K, ldx, ldw):
    for save in (None, BF16, E4M3):
        for count in (0, 4):
            assert call(lib, M, N, K, rank, count, save, ldx, ldw)[0] == 0, (save, count)
        assert call(lib, M, N, K, rank, 4, E4M3, ldx, ldw, short=1 << 40)[0] == -13


def test_workspace_size_refusals(lib):
    size, x, w = lib.hg_linear_adapters_workspace_size, mat(0, 64), mat(1, 64)
    assert size(4, 8, 64, 16, x, w) == 256 and size(0, 8, 64, 16, x, w) == 0 and size(4, 8, 0, 16, x, w) == 0
    assert size(-1, 8, 64, 999, None, None) == -1 and size(4, -1, 64, 999, x, w) == -2 and size(4, 8, -1, 9, x, w) == -3
    assert size(4, 8, 64, 257, x, w) == -4 and size(4, 8, 64, -1, x, w) == -4
    assert size(4, 8, 64, 16, None, w) == -5 and size(4, 8, 64, 16, x, mat(1, 64, F16)) == -6


@pytest.mark.parametrize("M,N,K", [(8192, 4096, 4096), (7840, 2816, 5560), (3001, 3026, 148), (64, 8224, 512)])
@pytest.mark.parametrize("kw", [dict(rank=17, count=0), dict(rank=16, count=0), dict(rank=0, count=4)])
def test_without_adapters_the_layer_is_cut_alike(lib, M, N, K, kw):
    """Whatever the rank of adapters that there are none of, and in the workspace that the rank asks for."""
    X, W, Y = mat(0, K), mat(1, K), mat(2, N)
    assert lib.hg_linear(4, M, N, K, X, W, None, None, Y, None, 9 * SPACE, lib.hg_linear_workspace_size(M, N, K, X, W), None) == 0
    alone = lib.plan_launches()
    X, W = mat(0, K), mat(1, K)
    L = adapters.Adapters(5 * SPACE, None, 6 * SPACE, K, 0, 7 * SPACE, max(1, kw["rank"]), 0, kw["count"], kw["rank"], BF16)
    work = lib.hg_linear_adapters_workspace_size(M, N, K, kw["rank"], X, W)
    assert lib.hg_linear_adapters(4, M, N, K, X, W, None, None, Y, None, L, 9 * SPACE, work, None) == 0
    assert lib.plan_launches() == alone


@pytest.mark.parametrize("M,N,K", [(100, 512, 512), (1000, 4096, 256), (8192, 4096, 4096), (32, 7412, 11584), (3, 512, 512), (300, 260, 4000)])
@pytest.mark.parametrize("rank", [1, 8, 11, 16, 24, 64, 256])
def test_three_numbers_for_an_fp32_result(lib, M, N, K, rank):
    """Rows of T for bf16 products with Y in fp32, in the workspace that is the same for any Y."""
    X, W = mat(0, K), mat(1, K)
    L = adapters.Adapters(5 * SPACE, None, 6 * SPACE, K, rank * K, 7 * SPACE, rank, N * rank, 4, rank, BF16)
    work = lib.hg_linear_adapters_workspace_size(M, N, K, rank, X, W)
    up = -(-rank // 8) * 8
    for type, parts in ((F32, 3), (BF16, 2)):
        assert lib.hg_linear_adapters(0, M, N, K, X, W, None, None, mat(2, N, type), None, L, 9 * SPACE, work, None) == 0
        kernel, edge = lib.plan_launches().decode().split()[:2]
        if kernel != "rowwise":
            assert edge == "edge=%d" % (up if kernel == "shrink_wide" else -(-parts * up // 32) * 32)


@pytest.mark.parametrize("M,N,K", [(100, 512, 512), (1000, 4096, 256), (8192, 4096, 4096), (8192, 4096, 4095), (3, 512, 512), (300, 260, 4000)])
@pytest.mark.parametrize("rank", [1, 16, 33])
def test_one_workspace_in_fp16(lib, M, N, K, rank):
    """With room for what fp16 does not reach, for Y and Z of either type."""
    X, W = mat(0, K, F16), mat(1, K, F16)
    L = adapters.Adapters(5 * SPACE, None, 6 * SPACE, K, rank * K, 7 * SPACE, rank, N * rank, 4, rank, F16)
    work = lib.hg_linear_adapters_workspace_size(M, N, K, rank, X, W)
    up = -(-rank // 8) * 8
    rows = M * up * 4 if M == 3 else M * up * 4 + M * -(-2 * up // 32) * 64
    assert work >= rows
    for y in (F16, F32):
        for z in (None, F16, E4M3):
            Z = None if z is None else mat(3, N, z)
            assert lib.hg_linear_adapters(0, M, N, K, X, W, None, None, mat(2, N, y), Z, L, 9 * SPACE, work, None) == 0
            assert lib.hg_linear_adapters(0, M, N, K, X, W, None, None, mat(2, N, y), Z, L, 9 * SPACE, rows - 256, None) == -13
