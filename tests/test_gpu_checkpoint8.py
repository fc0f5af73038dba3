"""8-bit checkpoints (hg_checkpoint8_write / _read) against their definition:
codes, scale bytes and values read back are exact, so they are compared for
equality (NaN codes by being NaN)."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float16, torch.bfloat16]


def matrix(seed, M, N, t, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N + pad, generator=g) * torch.exp2(torch.randint(-12, 10, (M, 1), generator=g).float())
    x[torch.rand(M, N + pad, generator=g) < 0.02] = 0.0
    return x.to(t)[:, :N]


def write(hg, X, cpad=0, spad=0):
    M, N = X.shape
    nb = -(-N // 32)
    codes = torch.full((M, N + cpad), 0x5a, dtype=torch.uint8, device=DEV)
    scales = torch.full((M, nb + spad), 0x5a, dtype=torch.uint8, device=DEV)
    hg.checkpoint8_write(X, codes[:, :N], scales[:, :nb])
    torch.cuda.synchronize()
    assert (codes[:, N:] == 0x5a).all() and (scales[:, nb:] == 0x5a).all()
    return codes[:, :N], scales[:, :nb]


def same(a, b):
    return ((a == b) | (a.isnan() & b.isnan())).all()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,N,pad", [(1, 1, 0), (1, 32, 0), (3, 33, 0), (5, 31, 3), (17, 64, 8), (7, 250, 6),
                                     (130, 1000, 0), (33, 4099, 1)])
def test_round_trip(hg, M, N, pad, t):
    print(f"[check8] {M}x{N} pad {pad} {t}", flush=True)
    X = matrix(M + N, M, N, t, pad)
    Xd = X.to(DEV) if pad == 0 else torch.nn.functional.pad(X, (0, pad)).to(DEV)[:, :N]
    codes, scales = write(hg, Xd, cpad=pad, spad=pad)
    vals, want = ref.codes8(X)
    assert torch.equal(scales.cpu(), want)
    assert same(ref.values8(codes, scales), vals)
    back = torch.full((M, N + pad), 7.0, dtype=t, device=DEV)
    hg.checkpoint8_read(codes, scales, back[:, :N])
    torch.cuda.synchronize()
    assert same(back[:, :N].cpu().double(), vals) and (back[:, N:] == 7.0).all()


@pytest.mark.parametrize("t", TYPES)
def test_every_16_bit_value(hg, t):
    """All 2^16 patterns, as blocks of one value each (columns 1..31 zero), then 32 to a block."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(t)
    for X in (torch.nn.functional.pad(bits.view(-1, 1), (0, 31)).contiguous(), bits.view(2048, 32)):
        codes, scales = write(hg, X.to(DEV))
        vals, want = ref.codes8(X)
        assert torch.equal(scales.cpu(), want)
        got = ref.values8(codes, scales)
        assert same(got, vals)
        back = torch.empty_like(X, device=DEV)
        hg.checkpoint8_read(codes, scales, back)
        assert same(back.cpu().double(), vals)          # what a code stands for is exact in the type


def test_every_code_and_scale_read(hg):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).view(-1, 1).repeat(1, 8)
    want = ref.values8(codes, scales)
    want[255] = float("nan")
    for t in TYPES:
        out = torch.empty(256, 256, dtype=t, device=DEV)
        hg.checkpoint8_read(codes.to(DEV), scales.to(DEV), out)
        assert same(out.cpu().double(), want.to(t).double())
    f8 = codes.view(torch.float8_e4m3fn).to(DEV)        # the codes' other dtype
    out2 = torch.empty(256, 256, dtype=torch.bfloat16, device=DEV)
    hg.checkpoint8_read(f8, scales.to(DEV), out2)
    assert same(out2.double(), out.double())


def test_non_finite_elements_leave_their_block_alone(hg):
    X = torch.ones(2, 64, dtype=torch.bfloat16)
    X[0, 3], X[0, 5], X[0, 40] = float("inf"), float("nan"), float("-inf")
    codes, scales = write(hg, X.to(DEV))
    vals = ref.values8(codes, scales)
    assert vals[0, [3, 5, 40]].isnan().all()
    keep = torch.ones(2, 64, dtype=torch.bool)
    keep[0, [3, 5, 40]] = False
    assert (vals[keep] == 1).all()


def test_many_rows_past_one_grid(hg):
    """More threads' work than one launch holds: the grid-stride loop; offsets past 2^31 bytes of the matrix."""
    M, N = 70001, 16400
    X = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    X[-1] = torch.linspace(-3, 3, N, device=DEV).to(torch.bfloat16)
    X[M // 2, 5] = 1.5
    codes, scales = hg.checkpoint8_write(X, *hg.checkpoint8_empty(M, N, DEV))
    back = torch.full((M, N), 9.0, dtype=torch.bfloat16, device=DEV)
    hg.checkpoint8_read(codes, scales, back)
    want, _ = ref.codes8(X[-1:].cpu())
    assert same(back[-1:].cpu().double(), want) and float(back[M // 2, 5]) == 1.5
    assert int((back != 0).sum()) == int((want != 0).sum()) + 1
