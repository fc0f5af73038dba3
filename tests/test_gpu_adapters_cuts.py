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


@pytest.mark.parametrize("t,out", [(F16, F16), (BF16, F32)])
@pytest.mark.parametrize("size", [(1, 256, 512), (33, 512, 512), (66, 100, 24), (79, 70, 2010), (4106, 71, 5056), (8294, 457, 16)])
def test_residual_in_place(hg, size, t, out):
    """R is Y itself."""
    X, W, A, B, s, which = (x.to(DEV) for x in operands(*size, 16, 5, t, "single"))
    r = torch.randn(size[:2], generator=torch.Generator().manual_seed(2)).to(out).to(DEV)
    Y = r.clone()
    hg.linear_adapters(X, W, Y, which, A, B, scales=s, act=hg.ACT_SILU, residual=Y)
    y, _, ey, _ = expected(X, W, A, B, s, which, None, "silu", r)
    ref.check(Y, y.cpu(), ey.cpu(), "Y")


@pytest.mark.parametrize("size", [(1, 256, 512), (40, 512, 512), (300, 260, 4000), (4096, 4096, 64)])
@pytest.mark.parametrize("t", [F16, BF16])
def test_two_calls_at_once(hg, size, t):
    """On two streams, a workspace each, over and over: each gets its own results."""
    calls = []
    for seed in (0, 1):
        X, W, A, B, s, which = (x.to(DEV) for x in operands(*size, 16, 6, t, "single", seed=seed))
        want = hg.linear_adapters(X, W, torch.empty(size[:2], dtype=t, device=DEV), which, A, B, scales=s)
        calls.append((X, W, torch.empty_like(want), which, A, B, s, hg.linear_adapters_workspace(X, W, A), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for X, W, Y, which, A, B, s, work, want, stream in calls:
            with torch.cuda.stream(stream):
                hg.linear_adapters(X, W, Y, which, A, B, scales=s, work=work)
    torch.cuda.synchronize()
    for c in calls:
        assert torch.equal(c[2], c[8])


@pytest.mark.parametrize("size", [(1, 256, 512), (40, 512, 512), (300, 260, 400), (4096, 4096, 64)])
def test_numbers_that_are_no_adapter(hg, size):
    """Any number outside 0 .. count-1, the largest and smallest of 64 bits and those that are an adapter's in their low
    32 among them."""
    M = size[0]
    X, W, A, B, s, which = (x.to(DEV) for x in operands(*size, 16, 6, BF16, "single"))
    which = which.clamp(0, 5)
    none = torch.tensor([-1, 6, 1 << 32, (1 << 32) + 3, -(1 << 32), (1 << 63) - 1, -(1 << 63), 5 - (1 << 32), 1 << 31, -(1 << 31)],
                        device=DEV)
    at = torch.arange(0, M, 2, device=DEV)
    which[at] = none[at // 2 % 10]
    Y = torch.empty(size[:2], dtype=BF16, device=DEV)
    hg.linear_adapters(X, W, Y, which, A, B, scales=s)
    mine = torch.where((which >= 0) & (which < 6), which, -1)
    y, _, ey, _ = expected(X, W, A, B, s, mine, None, "none", None)
    ref.check(Y, y.cpu(), ey.cpu(), "Y")


@pytest.mark.parametrize("t,out", [(F16, F16), (BF16, F32)])
@pytest.mark.parametrize("size", [(3, 256, 512), (65, 512, 512), (333, 111, 777), (1000, 4096, 256), (4096, 4096, 64)])
@pytest.mark.parametrize("order", ["single", "runs"])
def test_the_largest_rank(hg, size, t, out, order):
    run(hg, *size, 256, 5, t, order, out)


@pytest.mark.parametrize("size", [(40, 512, 512), (300, 260, 400), (4096, 4096, 64)])
def test_one_b_for_all(hg, size):
    """B broadcast over the adapters, A their own, and the two together."""
    X, W, A, B, s, which = (x.to(DEV) for x in operands(*size, 16, 6, BF16, "single"))
    for a, b in ((A, B[:1].expand_as(B)), (A[:1].expand_as(A), B[:1].expand_as(B))):
        Y = torch.empty(size[:2], dtype=BF16, device=DEV)
        hg.linear_adapters(X, W, Y, which, a, b, scales=s)
        y, _, ey, _ = expected(X, W, a, b, s, which, None, "none", None)
        ref.check(Y, y.cpu(), ey.cpu(), "Y")
