"""The linear layer and its gradient on small integers, at sizes that cut the
products every way: each tile edge, no slices, all tiles in slices, only the
last round's tiles in slices, the row-wise form, both products of a gradient in
one launch or in two.

Sums of integers in -2 .. 2 stay below 2^24, so every fp32 sum is exact in any
order, and so is torch's fp32 product; what is rounded is rounded once.  The
workspace holds NaN before the call and the outputs are surrounded by a
pattern."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32

SHAPES = [(4133, 4365, 2048), (4133, 4365, 640), (2048, 2100, 1024), (2100, 1500, 1500), (1500, 1500, 6000),
          (3000, 6000, 4000), (700, 1000, 3000), (130, 260, 4096), (65, 64, 4096), (300, 4000, 8192),
          (1100, 1100, 4200), (2050, 2050, 300), (2050, 2050, 1000), (1300, 1400, 1600), (2000, 2000, 4096),
          (90, 8192, 512), (90, 70000, 64), (16, 4096, 16384), (33, 5000, 2056), (4096, 8192, 512), (8300, 520, 1000),
          (257, 4096, 8200), (1, 70000, 72), (64, 64, 1031), (2, 1 << 20, 8), (80, 24, 1 << 20)]


def ints(g, *shape):
    return torch.randint(-2, 3, shape, generator=g, device=DEV, dtype=torch.int8).float()


def room(M, N, t):
    buf = torch.full((M + 2, N + 8), -77.0, dtype=t, device=DEV)
    return buf, buf[1:M + 1, :N]


def around(buf, M, N):
    assert (buf[0] == -77).all() and (buf[M + 1] == -77).all() and (buf[:, N:] == -77).all()


def nan_work(need):
    return torch.full((need // 4 + 4,), float("nan"), device=DEV)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(hg, M, N, K):
    print(f"[cuts] forward {M}x{N}x{K}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(M * 31 + N * 7 + K)
    X, W, b, R = ints(g, M, K), ints(g, N, K), ints(g, N), ints(g, M, N)
    z = X @ W.t() + b
    for t, out, save8 in ((F16, F32, True), (BF16, BF16, False)):
        Xh, Wh = X.to(t), W.to(t)
        buf, Y = room(M, N, out)
        zbuf, Z = room(M, N, t)
        Z8 = hg.checkpoint8_empty(M, N, DEV)
        hg.linear(Xh, Wh, Y, bias=b, act=hg.ACT_RELU, residual=R.to(out), Z=Z8 if save8 else Z,
                  work=nan_work(hg.linear_workspace_size(Xh, Wh)))
        around(buf, M, N)
        assert torch.equal(Y, (z.relu() + R).to(out))
        if save8 and K < 1 << 20:                  # z is an integer below 2^11: exact in fp16
            assert float(z.abs().max()) < 2048
            want = hg.checkpoint8_write(z.half(), *hg.checkpoint8_empty(M, N, DEV))
            assert torch.equal(Z8[0], want[0]) and torch.equal(Z8[1], want[1])
        elif not save8:
            around(zbuf, M, N)
            assert torch.equal(Z, z.to(t))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gradient(hg, M, N, K):
    print(f"[cuts] gradient {M}x{N}x{K}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(M * 37 + N * 11 + K)
    X, W, dY, Z = ints(g, M, K), ints(g, N, K), ints(g, M, N), ints(g, M, N)
    dw0, db0 = ints(g, N, K), ints(g, N)
    dz = torch.where(Z > 0, dY, 0.0)
    dx, dw, db = dz @ W, dz.t() @ X, dz.sum(0)
    for t, wt, acc, want in ((F16, F32, False, "xwb"), (BF16, F32, True, "xwb"), (BF16, BF16, False, "x"),
                             (F16, F16, False, "w")):
        Xh, Wh, dYh, Zh = X.to(t), W.to(t), dY.to(t), Z.to(t)
        xb, dX = room(M, K, t)
        wb, dW = room(N, K, wt)
        dB = db0.clone()
        if acc:
            dW.copy_(dw0)
        hg.linear_grad(dYh, Wh, Xh, Z=Zh, act=hg.ACT_RELU, dX=dX if "x" in want else None,
                       dW=dW if "w" in want else None, dbias=dB if "b" in want else None, accumulate=acc,
                       work=nan_work(hg.linear_grad_workspace_size(dYh, Wh, Xh)))
        around(xb, M, K)
        around(wb, N, K)
        if "x" in want:
            assert torch.equal(dX, dx.to(t))
        if "w" in want:
            assert torch.equal(dW, (dw + dw0 if acc else dw).to(wt))
        if "b" in want:
            assert torch.equal(dB, db + db0 if acc else db)


@pytest.mark.parametrize("M,N,K", [(2050, 2050, 1000), (4133, 4365, 2048), (300, 4000, 8192)])
def test_cut_products_in_place_and_again(hg, M, N, K):
    """Slices with the residual in place, twice on one workspace: nothing of the first call is left in the second."""
    g = torch.Generator(device=DEV).manual_seed(3)
    X, W, R = ints(g, M, K).to(F16), ints(g, N, K).to(F16), ints(g, M, N)
    Y = R.clone()
    work = nan_work(hg.linear_workspace_size(X, W))
    hg.linear(X, W, Y, residual=Y, work=work)
    hg.linear(X, W, Y, residual=Y, work=work)
    assert torch.equal(Y, 2 * (X.float() @ W.float().t()) + R)


def test_offsets_past_32_bits(hg):
    """Every matrix with rows so far apart that its last element lies past 2^32 bytes."""
    M, N, K, ld = 70000, 72, 136, 32768
    g = torch.Generator(device=DEV).manual_seed(4)
    X, W, dY, Z = ints(g, M, K), ints(g, N, K), ints(g, M, N), ints(g, M, N)

    def far(x, t):
        big = torch.empty(M, ld, dtype=t, device=DEV)
        v = big[:, 8:8 + x.shape[1]]
        v.copy_(x)
        return v
    Xh, dYh, Zh = far(X, F16), far(dY, F16), far(Z, F16)
    Y, R = far(dY, F32), far(Z, F32)
    hg.linear(Xh, W.to(F16), Y, residual=R, act=hg.ACT_RELU, Z=Zh)
    z = X @ W.t()
    assert torch.equal(Y, z.relu() + Z) and torch.equal(Zh, z.half())
    Zh.copy_(Z)
    dX, dW, db = far(X, F16), torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    hg.linear_grad(dYh, W.to(F16), Xh, Z=Zh, act=hg.ACT_RELU, dX=dX, dW=dW, dbias=db)
    dz = torch.where(Z > 0, dY, 0.0)
    assert torch.equal(dX, (dz @ W).half()) and torch.equal(dW, dz.t() @ X) and torch.equal(db, dz.sum(0))
    codes, scales = torch.empty(M, ld * 2, dtype=torch.uint8, device=DEV)[:, :K], torch.empty(M, 5, dtype=torch.uint8, device=DEV)
    hg.checkpoint8_write(Xh, codes, scales)
    back = hg.checkpoint8_read(codes, scales, far(Z[:, :1].expand(M, K), F16))
    assert torch.equal(back, Xh)                       # small integers are exact in e4m3
    hg.linear_grad(dYh, W.to(F16), (codes, scales), Z=Zh, act=hg.ACT_RELU, dW=dW, accumulate=True)
    assert torch.equal(dW, 2 * (dz.t() @ X))


@pytest.mark.parametrize("save", [None, "8"])
@pytest.mark.parametrize("K", [8, 248, 256, 264, 1280, 2048, 2056, 4352])
@pytest.mark.parametrize("N", [1, 16, 40, 4100, 8200, 16400])
def test_few_rows(hg, N, K, save):
    """Every count of rows that takes another form, sums that end inside a stage and are shorter or longer than the
    ring, more workgroups than compute units, NaN behind every row and below the last one; K = 4352 is 17 stages."""
    print(f"[cuts] few rows N={N} K={K} {save}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(N + K)
    big = torch.full((65, K + 8), float("nan"), dtype=F16, device=DEV)
    wide = torch.full((N + 1, K + 16), float("nan"), dtype=F16, device=DEV)
    W = wide[:N, :K]
    W.copy_(ints(g, N, K))
    for M in (1, 2, 15, 16, 17, 32, 33, 48, 64):
        big.fill_(float("nan"))
        X = big[:M, :K]
        X.copy_(ints(g, M, K))
        want = torch.mm(X.float(), W.float().t())
        buf, Y = room(M, N, F32)
        Z = hg.checkpoint8_empty(M, N) if save else None
        hg.linear(X, W, Y, Z=Z)
        assert torch.equal(Y, want), (M, N, K)
        around(buf, M, N)
        if save:
            assert want.abs().max() <= 2048               # exact in fp16
            codes, scales = hg.checkpoint8_write(want.to(F16), *hg.checkpoint8_empty(M, N))
            assert torch.equal(Z[0], codes) and torch.equal(Z[1], scales), (M, N, K)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N,K", [(65, 64, 1), (64, 65, 7), (80, 70, 63), (333, 1111, 777), (100, 130, 65), (129, 64, 191),
                                   (70, 333, 257), (128, 1024, 8191), (300, 257, 1537), (1000, 1000, 1001), (200, 64, 64)])
def test_rows_at_odd_addresses(hg, M, N, K, t):
    """Both operands at odd addresses and rows of odd length, sums of no, one and many whole stages, with slices and
    without, NaN behind every row; with everything that follows the product."""
    print(f"[cuts] odd {M}x{N}x{K} {t}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(M + N + K)

    def odd(rows, cols):
        ld = cols + 1 + cols % 2
        flat = torch.full((rows * ld + 1,), float("nan"), dtype=t, device=DEV)
        m = flat[1:].view(rows, ld)[:, :cols]
        return m.copy_(ints(g, rows, cols))

    X, W, b = odd(M, K), odd(N, K), ints(g, N)
    R = ints(g, M, N)
    z = torch.mm(X.float(), W.float().t()) + b
    assert z.abs().max() < 2 ** 24
    buf, Y = room(M, N, F32)
    zbuf, Z = room(M, N, t)
    hg.linear(X, W, Y, bias=b, act=1, residual=R, Z=Z)
    assert torch.equal(Y, z.clamp(min=0) + R) and torch.equal(Z, z.to(t))
    around(buf, M, N)
    around(zbuf, M, N)
    if K % 8 == 0:                                          # one operand at odd addresses, the other not
        hg.linear(X.contiguous(), W, Y, bias=b, act=1, residual=R)
        assert torch.equal(Y, z.clamp(min=0) + R)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("out", [F16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 130, 60000), (64, 2000, 5000), (33, 4100, 1928), (16, 40000, 200),
                                   (2, 33000, 136), (63, 64, 100000), (9, 8256, 1000), (5, 4111, 1931),
                                   (64, 2049, 3005)])
def test_weight_of_few_rows(hg, M, N, K, out, accumulate):
    """dW of few rows: runs of one and many tiles, a last one that is not whole, more strips than places."""
    print(f"[cuts] weight {M}x{N}x{K} {out} {accumulate}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    X, dY = ints(g, M, K), ints(g, M, N)
    buf, dW = room(N, K, out)
    old = ints(g, N, K)
    dW.copy_(old)
    db = torch.empty(N, device=DEV)
    want = torch.mm(dY.t().contiguous(), X) + (old if accumulate else 0)
    assert want.abs().max() <= 2048                       # exact in fp16
    t = F16 if out is F16 else BF16
    hg.linear_grad(dY.to(t), None, X.to(t), dW=dW, dbias=None if accumulate else db, accumulate=accumulate)
    assert torch.equal(dW.float(), want)
    around(buf, N, K)
    if not accumulate:
        assert torch.equal(db, dY.sum(0))


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("K", [1, 7, 9, 63, 65, 511, 513, 1023, 2049])
@pytest.mark.parametrize("N", [1, 40, 8211])
def test_few_rows_at_odd_elements(hg, N, K, t):
    """Rows of W, of X or of both at odd elements: odd bases, odd row lengths, NaN before, between and behind rows."""
    print(f"[cuts] few odd rows N={N} K={K} {t}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(N + K)

    def put(rows, cols, base, ld):
        flat = torch.full((rows * ld + base + 1,), float("nan"), dtype=t, device=DEV)
        return flat[base:base + rows * ld].view(rows, ld)[:, :cols].copy_(ints(g, rows, cols))

    odd, even = K + 1 + K % 2, K + 2 - K % 2
    W = [put(N, K, 1, odd), put(N, K, 0, odd), put(N, K, 1, even), put(N, K, 0, even)]
    for M in (1, 2, 16, 17, 33, 64):
        for i, X in enumerate((put(M, K, 0, even), put(M, K, 1, odd), put(M, K, 0, odd), put(M, K, 1, even))):
            want = torch.mm(X.float(), W[i].float().t())
            buf, Y = room(M, N, F32)
            hg.linear(X, W[i], Y)
            assert torch.equal(Y, want), (M, N, K, i)
            around(buf, M, N)
