"""hg_linear_adapters: Y = act(X·Wᵀ + bias + s_g·(X·A_gᵀ)·B_gᵀ) + R, g the row's
adapter, against 64 bits.

Bound, in the terms of linear_ref.py.  t = s_g·Σ x·a in fp32 is off by et =
|s_g|·(K + 3)·u32·Σ|x|·|a|.  As two numbers of X's type, each a rounding of what
the one before leaves, it is off by half(X's type)² of it more, in fp16 at least
2^-25; |t| + that bounds the two.  The sum of K products and at most 2·(rank + 7)
+ 32 more terms is off by (K + 2·rank + 48)·u32 of their magnitudes, and by
et·Σ|b|.  bias, act and R as linear_ref.linear's.
"""
import pytest
import torch

import linear_ref as ref
from test_gpu_linear import BF16, DEV, F16, F32, act_of, room, strided

pytestmark = pytest.mark.gpu
U32 = ref.U32


def operands(M, N, K, rank, count, t, order, seed=0, scales=True):
    g = torch.Generator().manual_seed(seed * 1000003 + M * 7919 + N * 31 + K + rank)
    X = torch.randn(M, K, generator=g).to(t)
    W = (torch.randn(N, K, generator=g) / max(K, 1) ** 0.5).to(t)
    A = (torch.randn(count, rank, K, generator=g) / max(K, 1) ** 0.5).to(t)
    B = (0.5 * torch.randn(count, N, rank, generator=g)).to(t)
    s = torch.rand(count, generator=g) + 0.5 if scales else None
    if order == "single":
        which = torch.randint(-1, count + 1, (M,), generator=g)
    elif order == "one":
        which = torch.full((M,), count - 1)
    elif order == "none":
        which = torch.full((M,), -1)
    else:
        which = torch.randint(-1, count, (M // 50 + 1,), generator=g).repeat_interleave(
            torch.randint(1, 150, (M // 50 + 1,), generator=g))
        which = torch.cat((which, which.new_full((M,), 0)))[:M]
    return X, W, A, B, s, which.long()


def expected(X, W, A, B, s, which, bias, name, R):
    """(Y, Z, bound of Y, bound of Z) before the last rounding."""
    K, rank, count, t = X.shape[1], A.shape[1], A.shape[0], X.dtype
    x, w = X.double(), W.double()
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    ez = torch.zeros_like(z)
    for g in range(count):
        rows = (which == g).nonzero()[:, 0]
        a, b, f = A[g].double(), B[g].double(), 1.0 if s is None else float(s[g])
        v, size = f * (x[rows] @ a.t()), abs(f) * (x[rows].abs() @ a.abs().t())
        e = (K + 3) * U32 * size
        e = e + ref.half(t) ** 2 * (v.abs() + e) + (2.0 ** -25 if t == F16 else 0.0)
        z[rows] += v @ b.t()
        mag[rows] += (v.abs() + e) @ b.abs().t()
        ez[rows] = e @ b.abs().t()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ez = ez + (K + 2 * rank + 48) * U32 * mag
    y = ref.act(z, name)
    ey = 1.13 * ez + (z.abs() + ez) * 2.0 ** -20
    if R is not None:
        y = y + R.double()
        ey = ey + U32 * (y.abs() + ey)
    return y, z, ey, ez


def stack(x, pad, shift=0):
    """A (G, rows, cols) stack on the device, rows cols + pad apart, NaN between them."""
    G, rows, cols = x.shape
    buf = torch.full((G * (rows + 1) * (cols + pad) + shift,), float("nan"), dtype=x.dtype, device=DEV)
    v = buf[shift:].view(G, rows + 1, cols + pad)[:, :rows, :cols]
    v.copy_(x)
    return v


def case(hg, M, N, K, rank, count, t=BF16, order="runs", name="none", bias=False, R=False, out=None, save=None, pad=0,
         shift=0, apad=0, opad=0, scales=True, seed=0):
    print(f"[adapters] M={M} N={N} K={K} rank={rank} count={count} {t} {order} {name} out={out} save={save} pad={pad} "
          f"shift={shift} apad={apad}", flush=True)
    X, W, A, B, s, which = operands(M, N, K, rank, count, t, order, seed, scales)
    g = torch.Generator().manual_seed(seed + 5)
    b = torch.randn(N, generator=g) if bias else None
    r = torch.randn(M, N, generator=g).to(out or t) if R else None
    Y, around = room(M, N, out or t, opad)
    Z = hg.checkpoint8_empty(M, N, DEV) if save == 8 else torch.empty(M, N, dtype=t, device=DEV) if save else None
    got = hg.linear_adapters(strided(X, pad, shift), strided(W, pad, shift), Y, which.to(DEV), stack(A, apad, shift),
                             stack(B, apad, shift), scales=None if s is None else s.to(DEV),
                             bias=None if b is None else b.to(DEV), act=act_of(hg, name),
                             residual=None if r is None else r.to(DEV), Z=Z)
    assert got is Y
    torch.cuda.synchronize()
    around()
    y, z, ey, ez = expected(X, W, A, B, s, which, b, name, r)
    ref.check(Y, y, ey, "Y")
    if save == 16:
        ref.check(Z, z, ez, "Z")
    elif save == 8:
        v = ref.values8(*Z)
        step = torch.exp2(Z[1].cpu().double() - 127).repeat_interleave(ref.BLOCK, 1)[:, :N]
        assert ((v - z).abs() <= ez + torch.maximum(2.0 ** -4 * (z.abs() + ez), 2.0 ** -10 * step)).all()


# few rows: through LDS, through registers, at odd elements
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64])
@pytest.mark.parametrize("N,K,rank,pad,shift,order", [
    (256, 512, 16, 0, 0, "single"), (250, 2048, 8, 8, 0, "one"), (100, 333, 9, 1, 0, "single"), (65, 72, 64, 0, 1, "runs"),
    (1000, 64, 1, 0, 0, "single"), (33, 8, 100, 0, 0, "single"),
])
def test_few_rows(hg, t, M, N, K, rank, pad, shift, order):
    case(hg, M, N, K, rank, 5, t, order, pad=pad, shift=shift, bias=M % 2 == 0)


@pytest.mark.parametrize("M,N,K", [(1, 16384, 4096), (16, 9000, 2048), (40, 8200, 256), (64, 8224, 512)])
def test_few_rows_of_wide_weights(hg, M, N, K):
    """32 rows of W in a workgroup."""
    case(hg, M, N, K, 16, 8, BF16, "single")


# 64×64 tiles, the same at any address, 128×128, slices, 256×256, with rows and columns that do not fill them
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N,K,rank,count,order,kw", [
    (65, 512, 512, 16, 5, "single", {}), (333, 111, 777, 9, 5, "single", dict(name="silu", bias=True)),
    (300, 260, 4000, 16, 3, "runs", dict(R=True, out=F32)), (700, 900, 640, 40, 4, "runs", dict(pad=8, apad=8)),
    (600, 1000, 100, 7, 64, "single", dict(save=8)), (1030, 2060, 131, 32, 6, "runs", dict(pad=1, opad=3)),
    (2048, 4096, 128, 17, 3, "runs", dict(bias=True, name="gelu")), (200, 300, 320, 256, 2, "single", {}),
    (1000, 1000, 200, 16, 1, "one", dict(scales=False, save=16)), (512, 512, 64, 16, 3, "none", {}),
])
def test_tiles(hg, t, M, N, K, rank, count, order, kw):
    case(hg, M, N, K, rank, count, t, order, **kw)


@pytest.mark.parametrize("M,N,K,rank,count,order,kw", [
    (4096, 4096, 64, 16, 4, "runs", {}), (3001, 5003, 128, 8, 300, "single", dict(out=F32)),
    (4000, 4000, 200, 32, 3, "runs", dict(R=True, name="gelu_tanh", save=16)), (2500, 4400, 264, 64, 2, "one", {}),
    (4096, 4096, 72, 24, 40, "single", dict(apad=1, shift=1)), (4100, 4200, 64, 16, 4, "none", dict(bias=True, save=8)),
])
@pytest.mark.parametrize("t", [F16, BF16])
def test_large_tiles(hg, t, M, N, K, rank, count, order, kw):
    case(hg, M, N, K, rank, count, t, order, **kw)


@pytest.mark.parametrize("M,N,K,rank", [(7, 40, 0, 16), (5, 64, 64, 0), (0, 64, 64, 16), (5, 0, 64, 16), (1, 1, 1, 1)])
def test_empty_and_smallest(hg, M, N, K, rank):
    case(hg, M, N, K, rank, 3, order="single", bias=True)


@pytest.mark.parametrize("M,N,K,rank", [(16, 256, 512, 16), (300, 256, 512, 16), (300, 256, 512, 9), (4096, 4096, 64, 16)])
@pytest.mark.parametrize("t", [F16, BF16])
def test_what_is_not_finite_stays_with_its_request(hg, t, M, N, K, rank):
    """Neither a row of X nor an adapter's A or B that holds a NaN or an infinity changes other requests' rows, and its
    own do not come out finite where it enters."""
    X, W, A, B, s, which = operands(M, N, K, rank, 6, t, "single")
    which[:] = torch.arange(M) % 5
    which[M // 2] = 5
    run = lambda: hg.linear_adapters(X.to(DEV), W.to(DEV), torch.empty(M, N, dtype=t, device=DEV), which.to(DEV),  # noqa: E731
                                     A.to(DEV), B.to(DEV), scales=s.to(DEV)).cpu()
    want = run()
    X[3, 5] = float("nan")
    A[1, 2 % rank, 3] = float("inf")
    B[2, 7, rank - 1] = float("nan")
    B[5, 11, 0] = float("inf")
    got = run()
    clean = (which != 1) & (which != 2) & (which != 5)
    clean[3] = False
    assert torch.equal(got[clean], want[clean])
    assert got[3].isnan().all() and not got[which == 1].isfinite().any()
    mine = got[which == 2]
    assert mine[:, 7].isnan().all() and not got[which == 5][:, 11].isfinite().any()


@pytest.mark.parametrize("M,N,K,rank", [(64, 256, 512, 16), (300, 256, 512, 16), (4096, 4096, 64, 16)])
def test_a_row_does_not_depend_on_the_others(hg, M, N, K, rank):
    """The same row beside other rows, in another place of its tile's adapters: the same bits."""
    X, W, A, B, s, which = (x.to(DEV) if x is not None else None for x in operands(M, N, K, rank, 6, BF16, "single"))
    X[M - 1], which[M - 1] = X[0], which[0].clamp(0, 5)
    which[0] = which[M - 1]
    Y = hg.linear_adapters(X, W, torch.empty(M, N, dtype=BF16, device=DEV), which, A, B, scales=s)
    close = (Y[0].double() - Y[M - 1].double()).abs() <= 2 * ref.half(BF16) * Y[0].double().abs() + 2.0 ** -12
    assert close.all()
    again = hg.linear_adapters(X, W, torch.empty(M, N, dtype=BF16, device=DEV), which, A, B, scales=s)
    assert torch.equal(Y, again)


@pytest.mark.parametrize("M,N,K", [(3, 512, 512), (200, 512, 512), (4096, 4096, 64)])
def test_graph(hg, M, N, K):
    """Captured and replayed with other rows, adapters and work between the replays."""
    X, W, A, B, s, which = (x.to(DEV) for x in operands(M, N, K, 16, 6, BF16, "runs"))
    Y, eager = (torch.empty(M, N, dtype=BF16, device=DEV) for _ in range(2))
    work = hg.linear_adapters_workspace(X, W, A)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        hg.linear_adapters(X, W, Y, which, A, B, scales=s, work=work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hg.linear_adapters(X, W, Y, which, A, B, scales=s, work=work)
    for i in range(4):
        X.copy_(torch.randn(M, K, device=DEV))
        which.copy_(torch.randint(-1, 6, (M,), device=DEV))
        Y.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        hg.linear_adapters(X, W, eager, which, A, B, scales=s)
        assert torch.equal(Y, eager), i


def test_another_stream(hg):
    X, W, A, B, s, which = (x.to(DEV) for x in operands(50, 300, 512, 16, 6, F16, "single"))
    want = hg.linear_adapters(X, W, torch.empty(50, 300, dtype=F16, device=DEV), which, A, B, scales=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = hg.linear_adapters(X, W, torch.empty(50, 300, dtype=F16, device=DEV), which, A, B, scales=s)
        torch.cuda.current_stream().synchronize()
    assert torch.equal(got, want)


def test_adapters_past_32_bits(hg):
    """Adapters 2^31 elements apart."""
    M, N, K, rank = 20, 64, 64, 8
    X, W, A, B, s, which = operands(M, N, K, rank, 3, BF16, "single")
    gap = (1 << 30) + 1000
    big = torch.zeros(2 * gap + 4096, dtype=BF16, device=DEV)
    a, b = big.as_strided((3, rank, K), (gap, K, 1)), big[1000:].as_strided((3, N, rank), (gap, rank, 1))
    a.copy_(A)
    b.copy_(B)
    Y = torch.empty(M, N, dtype=BF16, device=DEV)
    hg.linear_adapters(X.to(DEV), W.to(DEV), Y, which.to(DEV), a, b, scales=s.to(DEV))
    y, _, ey, _ = expected(X, W, A, B, s, which, None, "none", None)
    ref.check(Y, y, ey, "Y")


def test_without_adapters_it_is_the_layer(hg):
    for M in (5, 300):
        X, W, A, B, s, which = (x.to(DEV) for x in operands(M, 200, 128, 16, 3, BF16, "none"))
        want = hg.linear(X, W, torch.empty(M, 200, dtype=BF16, device=DEV))
        for a, b, f in ((A, B, s), (A[:0], B[:0], s[:0]), (A[:, :0], B[:, :, :0], s)):
            got = hg.linear_adapters(X, W, torch.empty(M, 200, dtype=BF16, device=DEV), which, a, b, scales=f)
            assert torch.equal(got, want)


def test_training_an_adapter_with_the_layer(hg):
    """One adapter's product as two layers, and its gradients: what the header says an adapter is trained with."""
    X, W, A, B, s, which = operands(300, 200, 256, 16, 1, F16, "one", scales=False)
    x, w, a, b = (v.to(DEV) for v in (X, W, A[0], B[0]))
    new = lambda *shape, t=F16: torch.empty(*shape, dtype=t, device=DEV)  # noqa: E731
    t = hg.linear(x, a, new(300, 16))
    y = hg.linear(t, b, new(300, 200, t=F32), residual=hg.linear(x, w, new(300, 200, t=F32)))
    both = hg.linear_adapters(x, w, new(300, 200, t=F32), which.to(DEV), A.to(DEV), B.to(DEV))
    ty = X.double() @ A[0].double().t()
    # the two differ by the rounding of t to fp16 and by fp32 sums
    lim = (ref.half(F16) * 1.01) * ty.abs() @ B[0].double().abs().t() + 2.0 ** -12
    assert ((y - both).cpu().double().abs() <= lim).all()
    dy = torch.randn(300, 200, generator=torch.Generator().manual_seed(1)).to(F16)
    dt, db, _ = hg.linear_grad(dy.to(DEV), b, t, dX=new(300, 16), dW=new(200, 16, t=F32))
    _, da, _ = hg.linear_grad(dt, a, x, dW=new(16, 256, t=F32))
    gt = ref.grads(dy, B[0], t.cpu(), torch.zeros(300, 200), "none")
    ref.check(dt, *gt["dX"], "dT")
    ref.check(db, *gt["dW"], "dB")
    ref.check(da, *ref.grads(dt.cpu(), A[0], X, torch.zeros(300, 16), "none")["dW"], "dA")


def test_one_a_for_all(hg):
    """A broadcast over the adapters, B their own."""
    M, N, K, rank = 70, 96, 128, 16
    X, W, A, B, s, which = operands(M, N, K, rank, 4, BF16, "single")
    A = A[:1].expand(4, rank, K)
    Y = torch.empty(M, N, dtype=BF16, device=DEV)
    hg.linear_adapters(X.to(DEV), W.to(DEV), Y, which.to(DEV), A[:1].to(DEV).expand(4, rank, K), B.to(DEV), scales=s.to(DEV))
    y, _, ey, _ = expected(X, W, A, B, s, which, None, "none", None)
    ref.check(Y, y, ey, "Y")


@pytest.mark.parametrize("M", [1, 9])
def test_a_decoding_step(hg, M):
    """What a server runs for the next tokens: a projection with the requests' adapters onto the residual stream, the
    head, the most probable tokens; captured, replayed with other requests."""
    from test_gpu_logprobs import close, order
    from test_gpu_logprobs import expected as distribution
    K, V, rank, count, k = 256, 3001, 16, 5, 6
    X, W, A, B, s, which = (x.to(DEV) for x in operands(M, K, K, rank, count, BF16, "single"))
    g = torch.Generator().manual_seed(3)
    head = (torch.randn(V, K, generator=g) / 8).to(BF16).to(DEV)
    h, stream = (torch.randn(M, K, generator=g).to(BF16).to(DEV) for _ in range(2))
    logits = torch.empty(M, V, dtype=F32, device=DEV)
    entropy, top = torch.empty(M, device=DEV), (torch.empty(M, k, dtype=torch.int64, device=DEV), torch.empty(M, k, device=DEV))
    work, hwork = hg.linear_adapters_workspace(X, W, A), hg.linear_workspace(h, head)
    pwork = hg.logprobs_workspace(logits, k)

    def step():
        hg.linear_adapters(X, W, h, which, A, B, scales=s, residual=stream, work=work)
        hg.linear(h, head, logits, work=hwork)
        hg.logprobs(logits, entropy=entropy, top=top, work=pwork)

    with torch.cuda.stream(torch.cuda.Stream()):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x = torch.randn(M, K, generator=g).to(BF16)
        w = torch.randint(-1, count, (M,), generator=g)
        X.copy_(x)
        which.copy_(w)
        graph.replay()
        torch.cuda.synchronize()
        y, _, ey, _ = expected(x, W.cpu(), A.cpu(), B.cpu(), s.cpu(), w, None, "none", stream.cpu())
        ref.check(h, y, ey, "h")
        z, _, ez, _ = ref.linear(h.cpu(), head.cpu())
        ref.check(logits, z, ez, "logits")
        v, b = distribution(logits.cpu(), 1.0)
        ids = order(logits.cpu(), k)
        assert torch.equal(top[0].cpu(), ids)
        close(top[1], v["logp"].gather(1, ids), b["logp"].gather(1, ids), "top")
        close(entropy, v["entropy"][:, 0], b["entropy"][:, 0], "entropy")


# rows of one adapter gathered from 256: fewer and more adapters than rows, more than 16 rows of one, blocks that end early
@pytest.mark.parametrize("K", [72, 75])
@pytest.mark.parametrize("M,rank,count", [(777, 16, 1), (777, 16, 2), (256, 33, 16), (257, 16, 255), (511, 5, 256), (512, 16, 257),
                                          (777, 64, 1000), (1025, 16, 70000)])
def test_rows_in_no_order(hg, M, rank, count, K):
    case(hg, M, 64, K, rank, count, BF16, "single")


def test_every_place_in_a_block(hg):
    """A lone adapter's row at every place of 256, the others' without one or of another."""
    M, N, K, rank = 256, 16, 64, 8
    X, W, A, B, s, _ = operands(M, N, K, rank, 3, F16, "single")
    dev = [x.to(DEV) for x in (X, W, A, B, s)]
    for other in (-1, 1):
        which = [torch.full((M,), other).index_fill(0, torch.tensor([i]), 2) for i in range(0, M, 5)]
        for w in which:
            Y = torch.empty(M, N, dtype=F16, device=DEV)
            hg.linear_adapters(dev[0], dev[1], Y, w.to(DEV), dev[2], dev[3], scales=dev[4])
            y, _, ey, _ = expected(X, W, A, B, s, w, None, "none", None)
            ref.check(Y, y, ey, "Y")


def test_more_blocks_than_a_launch_takes(hg):
    """2^25 rows and some, blocks without an adapter among them: integers, exact."""
    M, K, N, count = (1 << 25) + 300, 8, 8, 3
    g = torch.Generator(device=DEV).manual_seed(3)
    few = lambda *shape: torch.randint(-1, 2, shape, generator=g, device=DEV).to(BF16)  # noqa: E731
    X, W, A, B = few(M, K), few(N, K), few(count, 1, K), few(count, N, 1)
    at = torch.arange(M, device=DEV)
    which = at * 2654435761 % 1000003 % 5 - 1
    which[at // 256 % 3 == 1] = -1
    Y = hg.linear_adapters(X, W, torch.empty(M, N, dtype=BF16, device=DEV), which, A, B)
    torch.cuda.synchronize()
    step = 1 << 23
    for i in range(0, M, step):
        x, w = X[i:i + step].float(), which[i:i + step]
        y = sum(x[:, k, None] * W[:, k].float() for k in range(K))
        for a in range(count):
            t = (x * A[a, 0].float()).sum(1) * (w == a)
            y += t[:, None] * B[a, :, 0].float()
        assert torch.equal(Y[i:i + step].float(), y)


# rows of many adapters in 128×128 tiles: rows of one that are more than 16 of a wave's, ranks of several steps, edges
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N,K,rank,count", [(1000, 4096, 256, 64, 64), (1000, 4096, 264, 20, 5), (901, 4001, 128, 100, 7),
                                              (1024, 2048, 1024, 8, 4), (700, 5000, 64, 3, 1000), (901, 4001, 128, 32, 7),
                                              (300, 200, 64, 72, 40), (1100, 2500, 128, 200, 9), (333, 111, 77, 256, 33)])
def test_many_adapters_in_a_tile(hg, t, M, N, K, rank, count):
    case(hg, M, N, K, rank, count, t, "single")


def test_infinities_stay_in_their_rows_among_many(hg):
    """What is not finite in some adapters' B and in some rows of X, rows of many adapters side by side."""
    for M, N, rank in ((300, 200, 16), (1000, 4096, 16), (300, 200, 64), (1000, 4096, 64)):
        X, W, A, B, s, which = operands(M, N, 64, rank, 12, BF16, "single")
        Y = []
        for bad in (False, True):
            x, b = X.clone(), B.clone()
            if bad:
                b[3, 5, 2], b[7, 100, 0], x[17, 3] = float("inf"), float("nan"), float("-inf")
            y = torch.empty(M, N, dtype=BF16, device=DEV)
            Y.append(hg.linear_adapters(x.to(DEV), W.to(DEV), y, which.to(DEV), A.to(DEV), b.to(DEV), scales=s.to(DEV)).cpu())
        touched = (which == 3) | (which == 7) | (torch.arange(M) == 17)
        assert torch.equal(Y[0][~touched], Y[1][~touched])
        assert not Y[1][which == 3][:, 5].isfinite().any() and Y[1][which == 7][:, 100].isnan().all()


@pytest.mark.parametrize("M,N,rank,count,apad", [(300, 300, 60, 40, 0), (300, 300, 58, 40, 2), (1000, 4096, 30, 16, 4), (900, 4100, 100, 9, 6),
                                                 (1000, 4096, 33, 16, 1), (300, 300, 57, 9, 3)])
def test_ranks_cut_from_padded_rows(hg, M, N, rank, count, apad):
    """What lies between B's rows (NaN) is loaded with them in places and must not count."""
    case(hg, M, N, 64, rank, count, BF16, "single", apad=apad)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("K", [8, 128, 512, 4096, 4104, 6000])
def test_an_infinite_a_of_one_row(hg, t, K):
    """One row, one launch: an infinity at either end of a row of A gives infinities as in the formula, no NaN."""
    N, rank, count = 64, 9, 2
    X, W, A, B, _, which = operands(1, N, K, rank, count, t, "one", scales=False)
    X, B = X.abs() + 0.5, torch.where(B.abs() < 0.1, 0.1, B).to(t)
    X = X.to(t)
    for k in (K - 1, 0):
        a = A.clone()
        a[1, 3, k] = float("inf")
        Y = torch.empty(1, N, dtype=F32, device=DEV)
        hg.linear_adapters(X.to(DEV), W.to(DEV), Y, which.to(DEV), a.to(DEV), B.to(DEV))
        assert torch.equal(Y[0].cpu(), torch.where(B[1, :, 3] > 0, float("inf"), -float("inf")).float()), k


# W is zero, and A and B have one value a value of T and a column: T comes out alone, with nothing that a sum could hide.
# 64×64 tiles at any address, 64×64, 128×128, 256×256, slices of each, few rows in tiles.
PLANS = [(333, 111, 777), (100, 512, 512), (1000, 4096, 256), (4096, 4096, 64), (300, 260, 4000), (32, 7412, 11584)]


def alone(M, N, K, rank, count, t, order, a=1.0, b=1.0, spread=False):
    """(X, W, A, B, s, which, T in fp32 by column); a: A's values, b: B's; spread: rows of very different size."""
    X, _, _, _, s, which = operands(M, N, K, rank, count, t, order)
    g = torch.Generator().manual_seed(M + N + K + rank)
    if spread:
        X = (X * torch.exp2(torch.randint(-9, 6, (M, 1), generator=g).float())).to(t)
    A, B = torch.zeros(count, rank, K, dtype=t), torch.zeros(count, N, rank, dtype=t)
    at = torch.randint(0, K, (count, rank), generator=g)
    value = (a * torch.randn(count, rank, generator=g).clamp(-2, 2)).to(t)
    A.scatter_(2, at[:, :, None], value[:, :, None])
    B[:, torch.arange(N), torch.arange(N) % rank] = b
    T = torch.zeros(M, rank)
    for c in range(count):
        rows = which == c
        T[rows] = X[rows][:, at[c]].float() * value[c].float() * s[c]
    return X, torch.zeros(N, K, dtype=t), A, B, s, which, T[:, torch.arange(N) % rank]


@pytest.mark.parametrize("M,N,K", PLANS)
@pytest.mark.parametrize("rank", [1, 8, 16, 33, 60, 64])
@pytest.mark.parametrize("order,count", [("single", 40), ("runs", 3)])
def test_t_is_as_exact_as_an_fp32_result(hg, M, N, K, rank, order, count):
    """bf16 with Y in fp32: T as a sum of bf16 numbers loses nothing of its 24 bits."""
    X, W, A, B, s, which, T = alone(M, N, K, rank, count, BF16, order)
    Y = torch.empty(M, N, dtype=F32, device=DEV)
    hg.linear_adapters(X.to(DEV), W.to(DEV), Y, which.to(DEV), A.to(DEV), B.to(DEV), scales=s.to(DEV))
    assert torch.equal(Y.cpu(), T)


@pytest.mark.parametrize("M,N,K", [(40, 512, 512)] + PLANS)
@pytest.mark.parametrize("rank", [1, 8, 16, 33, 60, 64])
@pytest.mark.parametrize("order,count", [("single", 40), ("runs", 3)])
def test_values_of_t_past_fp16(hg, M, N, K, rank, order, count):
    """fp16: values of X·A_gᵀ past 65504, beside others of the same row within it, are finite as in the formula whatever
    the number of rows; what is infinite stays that, in its rows."""
    X, W, A, B, s, which, T = alone(M, N, K, rank, count, F16, order, a=30000.0, b=2.0 ** -14, spread=True)
    # (a few rows in runs may have small values alone)
    assert order == "runs" or ((T.abs() > 65520).any() and (T.abs() < 65504).any())
    bad = int(which.max())
    bad = bad if 0 < bad < count else -1
    if bad >= 0:
        A[bad, rank - 1, A[bad, rank - 1].float().abs().argmax()] = float("inf")
    Y = torch.empty(M, N, dtype=F32, device=DEV)
    hg.linear_adapters(X.to(DEV), W.to(DEV), Y, which.to(DEV), A.to(DEV), B.to(DEV), scales=s.to(DEV))
    got, want = Y.cpu().double(), T.double() * 2.0 ** -14
    mine = which == bad if bad >= 0 else torch.zeros(M, dtype=torch.bool)
    assert not got[mine][:, rank - 1::rank].isfinite().any()
    # two fp16 numbers are off by 2^-22 of T, or 2^-25; the product is exact, the sum an fp32 one
    lim = want.abs() * (2.0 ** -22 + 2.0 ** -23) + 2.0 ** -39
    assert ((got - want).abs() <= lim)[~mine].all()


@pytest.mark.parametrize("M,N,K", [(64, 256, 512), (300, 256, 512), (4096, 4096, 64)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_a_row_in_two_places(hg, M, N, K, out):
    """The same row beside other rows: both are the formula's within the bound (their last bits may differ)."""
    X, W, A, B, s, which = operands(M, N, K, 16, 6, BF16, "single")
    which[0] = 3
    X[M - 1], which[M - 1] = X[0], which[0]
    Y = hg.linear_adapters(*(x.to(DEV) for x in (X, W)), torch.empty(M, N, dtype=out, device=DEV),
                           *(x.to(DEV) for x in (which, A, B)), scales=s.to(DEV))
    two = [0, M - 1]
    y, _, ey, _ = expected(X[two], W, A, B, s, which[two], None, "none", None)
    ref.check(Y[two], y, ey, "Y")


@pytest.mark.parametrize("t", [F16, BF16])
def test_the_gradient_of_an_adapted_layer(hg, t):
    """What the header says of a backward pass: rows of one adapter at a time, the layer's dX and the adapter's added by the
    caller.  dX, dA and dB against the formula's and, in a direction each, against differences in 64 bits."""
    M, N, K, rank, count = 200, 96, 160, 16, 3
    X, W, A, B, _, which = operands(M, N, K, rank, count, t, "single", scales=False)
    dY = torch.randn(M, N, generator=torch.Generator().manual_seed(4)).to(t)
    new = lambda *shape, type=t: torch.empty(*shape, dtype=type, device=DEV)  # noqa: E731
    dx = hg.linear_grad(dY.to(DEV), W.to(DEV), None, dX=new(M, K))[0].cpu()
    dA, dB = torch.zeros(count, rank, K), torch.zeros(count, N, rank)
    for c in range(count):
        rows = (which == c).nonzero()[:, 0]
        x, dy, a, b = X[rows].to(DEV), dY[rows].to(DEV), A[c].to(DEV), B[c].to(DEV)
        T = hg.linear(x, a, new(len(rows), rank))
        dT, db, _ = hg.linear_grad(dy, b, T, dX=new(len(rows), rank), dW=new(N, rank, type=F32))
        more, da, _ = hg.linear_grad(dT, a, x, dX=new(len(rows), K), dW=new(rank, K, type=F32))
        dx[rows] = (dx[rows].float() + more.cpu().float()).to(t)
        dA[c], dB[c] = da.cpu(), db.cpu()

    def z(x, a, b):
        out = x @ W.double().t()
        for c in range(count):
            rows = which == c
            out[rows] += x[rows] @ a[c].t() @ b[c].t()
        return out

    x, w, a, b, dy, h = X.double(), W.double(), A.double(), B.double(), dY.double(), ref.half(t) * 1.01
    wx, ex = dy @ w, (N + 2) * U32 * (dy.abs() @ w.abs())
    eA, eB = torch.zeros(count, rank, K).double(), torch.zeros(count, N, rank).double()
    for c in range(count):
        rows = which == c
        xr, dr, T, dT = x[rows], dy[rows], x[rows] @ a[c].t(), dy[rows] @ b[c]
        sT, sd = xr.abs() @ a[c].abs().t(), dr.abs() @ b[c].abs()
        # T and dT: sums in fp32, rounded once (fp16: by 2^-25 at least)
        eT, ed = (v.abs() * h + 1.01 * (n + 2) * U32 * s + ref.tiny(t) for v, n, s in ((T, K, sT), (dT, N, sd)))
        eB[c] = dr.abs().t() @ eT + (M + 2) * U32 * (dr.abs().t() @ (T.abs() + eT))
        eA[c] = ed.t() @ xr.abs() + (M + 2) * U32 * ((dT.abs() + ed).t() @ xr.abs())
        ref.check(dB[c], dr.t() @ T, eB[c], "dB")
        ref.check(dA[c], dT.t() @ xr, eA[c], "dA")
        e = ed @ a[c].abs() + (rank + 2) * U32 * ((dT.abs() + ed) @ a[c].abs())
        # two matrices rounded each
        ex[rows] += e + h * (wx[rows].abs() + ex[rows] + (dT @ a[c]).abs() + e) + 2 * ref.tiny(t)
        wx[rows] += dT @ a[c]
    ref.check(dx, wx, ex, "dX")
    g = torch.Generator().manual_seed(9)
    # z is linear in each: differences are exact but for 64 bits' rounding
    for got, at, err in ((dx, 0, ex), (dA, 1, eA), (dB, 2, eB)):
        args = [x, a, b]
        way = torch.randn(args[at].shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + way, args[at] - way
        change = ((z(*up) - z(*down)) / 2 * dy).sum()
        last = ref.half(got.dtype) * (got.double().abs() + err) * 1.01 + ref.tiny(got.dtype)
        assert ((got.double() * way).sum() - change).abs() <= ((err + last) * way.abs()).sum() + 1e-9
