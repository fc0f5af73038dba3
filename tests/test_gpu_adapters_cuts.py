"""hg_linear_adapters at every way its product is cut (adapters_cuts.py): the adapters'
terms are added once, in whatever piece of a sum, and T is whole, also in a workspace
that holds NaN throughout.  Bounds: test_gpu_adapters.py."""
import pytest
import torch

import linear_ref as ref
from adapters_cuts import FEW_IN_TILES, ROW_BY_ROW, TILES
from test_gpu_adapters import BF16, DEV, F16, F32, alone, expected, operands, room

pytestmark = pytest.mark.gpu


def run(hg, M, N, K, rank, count, t, order, out, R=False):
    print(f"[adapters] M={M} N={N} K={K} rank={rank} {t} {order} out={out} R={R}", flush=True)
    X, W, A, B, s, which = (x.to(DEV) for x in operands(M, N, K, rank, count, t, order))
    which[-1] = count - 1
    r = torch.randn(M, N, generator=torch.Generator().manual_seed(1)).to(out).to(DEV) if R else None
    Y, around = room(M, N, out, 0)
    work = torch.full((hg.linear_adapters_workspace_size(X, W, A),), 255, dtype=torch.uint8, device=DEV)
    hg.linear_adapters(X, W, Y, which, A, B, scales=s, residual=r, work=work)
    around()
    y, _, ey, _ = expected(X, W, A, B, s, which, None, "none", r)
    ref.check(Y, y.cpu(), ey.cpu(), "Y")


@pytest.mark.parametrize("t,out,order,rank", [(F16, F16, "single", 24), (BF16, F32, "runs", 16), (F16, F32, "runs", 64),
                                              (BF16, BF16, "single", 16), (BF16, F32, "single", 9)])
@pytest.mark.parametrize("size", TILES)
def test_tiles(hg, size, t, out, order, rank):
    run(hg, *size, rank if TILES[size][0] < 256 or rank % 8 == 0 else 8, 6, t, order, out, R=rank == 16)


@pytest.mark.parametrize("t,out", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rank", [1, 9, 16, 24, 33])
@pytest.mark.parametrize("size", FEW_IN_TILES)
def test_few_rows_in_tiles(hg, size, t, out, rank):
    run(hg, *size, rank, 7, t, "single", out)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("rank", [1, 16, 64])
@pytest.mark.parametrize("size", ROW_BY_ROW)
def test_row_by_row(hg, size, t, rank):
    """32 rows of W in a workgroup."""
    run(hg, *size, rank, 7, t, "single", t)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("order,count", [("single", 40), ("runs", 3)])
@pytest.mark.parametrize("size", list(TILES) + list(FEW_IN_TILES))
def test_t_alone(hg, size, order, count, t):
    """W is zero and Y in fp32: T in bf16 numbers is whole, in fp16 numbers within 2^-22, past fp16 whole (B is 2^-14
    there)."""
    half = t == F16
    X, W, A, B, s, which, T = alone(*size, 16, count, t, order, a=30000.0 if half else 1.0, b=2.0 ** -14 if half else 1.0,
                                    spread=half)
    X, W, A, B, s, which = (x.to(DEV) for x in (X, W, A, B, s, which))
    Y = torch.empty(size[:2], dtype=F32, device=DEV)
    work = torch.full((hg.linear_adapters_workspace_size(X, W, A),), 255, dtype=torch.uint8, device=DEV)
    hg.linear_adapters(X, W, Y, which, A, B, scales=s, work=work)
    want = T.to(DEV).double() * (2.0 ** -14 if half else 1.0)
    lim = want.abs() * (2.0 ** -22 + 2.0 ** -23) + 2.0 ** -39 if half else 0.0
    assert ((Y.double() - want).abs() <= lim).all()
