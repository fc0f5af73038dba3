"""The sizes of adapters_cuts.py are cut as they are meant to be, for every rank that
they are run with (CPU only, as test_adapters_plan.py)."""
import ctypes
import os
import subprocess

import pytest

import half_precision_gemm_amd.layer as layer
from adapters_cuts import FEW_IN_TILES, ROW_BY_ROW, TILES

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
F16, BF16 = 0, 2


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("cut") / "cut.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "half_precision_gemm_amd", "csrc"),
                    os.path.join(HERE, "adapters_cut_stub.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).adapters_cut
    f.argtypes = [ctypes.c_int64] * 4 + [ctypes.POINTER(layer.Matrix)] * 2 + [ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]

    def cut(M, N, K, rank, type=BF16):
        X, W = (layer.Matrix(i << 44, K, 0, 0, type) for i in (1, 2))
        out = (ctypes.c_int64 * 6)()
        f(M, N, K, rank, X, W, 0, out)
        tile, whole, splits, copies, loose, blocks = out
        return (tile, "none" if splits == 1 else "some" if whole > 0 else "all",
                "loose" if loose else "copied" if copies else "direct", blocks)
    return cut


@pytest.mark.parametrize("type", [F16, BF16])
@pytest.mark.parametrize("size", list(TILES) + list(FEW_IN_TILES))
def test_tiles(cut, size, type):
    want = {**TILES, **FEW_IN_TILES}[size]
    ranks = (16, 24, 64) + ((1, 9, 33) if want[0] < 256 else ())
    assert {cut(*size, rank, type)[:3] for rank in ranks} == {want}
    assert (size[0] <= 64) == (size in FEW_IN_TILES)


@pytest.mark.parametrize("size", ROW_BY_ROW)
def test_row_by_row(cut, size):
    assert {(c[0], c[3]) for c in (cut(*size, rank) for rank in (1, 9, 16, 64))} == {(0, 2)}
    assert min(-(-size[0] // 16), 4) == ROW_BY_ROW[size]
