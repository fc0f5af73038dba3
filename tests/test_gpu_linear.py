"""hg_linear: Y = act(X·Wᵀ + bias) + R with the pre-activation saved in 16 or 8
bits, against 64 bits (linear_ref.py: definitions and bounds)."""
import ctypes

import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def act_of(hg, name):
    return getattr(hg, "ACT_" + name.upper())


def strided(x, pad, shift=0):
    """x on the device in rows of ld = columns + pad, `shift` elements past an aligned address, NaN around it."""
    M, N = x.shape
    buf = torch.full((M * (N + pad) + shift + 16,), float("nan"), dtype=x.dtype, device=DEV)
    v = buf[shift:shift + M * (N + pad)].view(M, N + pad)[:, :N]
    v.copy_(x)
    return v


def room(M, N, t, pad):
    """An output in rows of N + pad, and a check that nothing around it was written."""
    buf = torch.full((M + 2, N + pad), -77.0, dtype=t, device=DEV)
    out = buf[1:M + 1, :N]

    def untouched():
        assert (buf[0] == -77).all() and (buf[M + 1] == -77).all() and (buf[:, N:] == -77).all()
    return out, untouched


def case(hg, M, N, K, t=F16, name="none", bias=True, R=False, out=None, save=None, pad=0, shift=0, opad=0, seed=0,
         in_place=False, integers=False):
    print(f"[linear] M={M} N={N} K={K} {t} {name} bias={bias} R={R} out={out} save={save} pad={pad} shift={shift}",
          flush=True)
    g = torch.Generator().manual_seed(seed * 1000003 + M * 7919 + N * 31 + K)
    out = out or t
    if integers:
        X, W = (torch.randint(-2, 3, s, generator=g).to(t) for s in ((M, K), (N, K)))
        b = torch.randint(-3, 4, (N,), generator=g).float() if bias else None
        r = torch.randint(-3, 4, (M, N), generator=g).to(out) if R else None
    else:
        X = torch.randn(M, K, generator=g).to(t)
        W = (torch.randn(N, K, generator=g) / max(K, 1) ** 0.5 * 2).to(t)
        b = torch.randn(N, generator=g) if bias else None
        r = torch.randn(M, N, generator=g).to(out) if R else None
    Y, around = room(M, N, out, opad)
    Rd = None
    if R:
        if in_place:
            Y.copy_(r)
            Rd = Y
        else:
            Rd = strided(r, opad)
    Z, zaround = None, None
    if save == "16":
        Z, zaround = room(M, N, t, opad)
    elif save == "8":
        Z = tuple(v.fill_(0x33) for v in hg.checkpoint8_empty(M, N, DEV))
    Xd, Wd = strided(X, pad, shift), strided(W, pad, shift)
    need = hg.linear_workspace_size(Xd, Wd)
    work = torch.full((need // 2 + 8,), float("nan"), dtype=F16, device=DEV)
    hg.linear(Xd, Wd, Y, bias=None if b is None else b.to(DEV), act=act_of(hg, name), residual=Rd, Z=Z, work=work)
    torch.cuda.synchronize()
    around()
    y, z, ey, ez = ref.linear(X, W, b, name, r)
    if integers:
        assert torch.equal(Y.cpu(), y.to(out)) if name in ("none", "relu") else True
    ref.check(Y, y, ey, "Y")
    if save == "16":
        zaround()
        ref.check(Z, z, ez, "Z")
    elif save == "8":
        check_saved8(Z, z, ez, t)
    return Y


def check_saved8(pair, z, ez, t):
    """The scale is the one of the block's largest magnitude, up to the fp32 sum's error at a border; each value is
    within half a step of e4m3 at that scale (clamped at the fp16 limit)."""
    codes, scales = pair
    M, N = z.shape
    e = scales.cpu().double() - 127
    pad = -N % 32
    blk = lambda v: torch.nn.functional.pad(v, (0, pad)).view(M, -1, 32).amax(2)  # noqa: E731
    amax, err = blk(z.abs()), blk(ez)
    lo = -15 if t == F16 else -117
    assert ((amax <= 448 * torch.exp2(e) + err) | ((t == F16) & (e == 8))).all()
    assert ((amax > 448 * torch.exp2(e - 1) - err) | (e == lo)).all()
    s = torch.exp2(e).repeat_interleave(32, 1)[:, :N]
    vals = ref.values8(codes, scales)
    lim = ez + torch.maximum(2.0 ** -4 * (z.abs() + ez), 2.0 ** -10 * s)
    bad = ~((vals - z).abs() <= lim)
    assert not bad.any(), (int(bad.sum()), z[bad][:4], vals[bad][:4], lim[bad][:4])


SHAPES = [(1, 1, 1), (1, 64, 8), (1, 100, 64), (1, 4096, 512), (2, 33, 40), (3, 257, 1000), (5, 31, 7), (8, 512, 4096),
          (16, 96, 136), (17, 65, 72), (31, 130, 200), (33, 1000, 64), (64, 64, 64), (65, 63, 65), (100, 300, 520),
          (128, 256, 2048), (129, 129, 129), (250, 511, 333), (257, 260, 8), (300, 1030, 1024), (40, 48, 16384)]


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(hg, M, N, K, t):
    case(hg, M, N, K, t)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_integers_are_exact(hg, M, N, K):
    """Sums of small integers are exact in fp32: every product and every index shows."""
    case(hg, M, N, K, BF16, "relu", R=True, out=F32, integers=True)
    case(hg, M, N, K, F16, "none", bias=False, out=F32, integers=True, pad=3)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("M,N,K,t,out", [(1, 300, 256, BF16, BF16), (70, 130, 96, F16, F32), (200, 264, 320, BF16, F32),
                                         (19, 1024, 64, F16, F16)])
def test_activations(hg, M, N, K, t, out, name):
    case(hg, M, N, K, t, name, R=True, out=out, save="16", opad=8)
    case(hg, M, N, K, t, name, bias=False, out=out, save="8")


@pytest.mark.parametrize("save", [None, "16", "8"])
@pytest.mark.parametrize("M,N,K,pad,shift,opad", [(1, 250, 128, 0, 0, 0), (13, 77, 100, 5, 1, 3), (129, 200, 64, 8, 0, 4),
                                                  (70, 1001, 136, 0, 4, 1), (256, 512, 256, 64, 8, 16),
                                                  (7, 34, 24, 0, 3, 6)])
def test_strides_and_alignment(hg, M, N, K, pad, shift, opad, save):
    case(hg, M, N, K, F16, "silu", R=True, save=save, pad=pad, shift=shift, opad=opad)
    case(hg, M, N, K, BF16, "gelu", R=True, out=F32, save=save, pad=pad, shift=shift, opad=opad)


@pytest.mark.parametrize("M,N,K", [(1, 128, 64), (40, 48, 16384), (130, 260, 512), (64, 100, 33)])
@pytest.mark.parametrize("out", [F16, F32])
def test_residual_in_place(hg, M, N, K, out):
    case(hg, M, N, K, F16, "gelu_tanh", R=True, out=out, in_place=True, opad=5)


def test_empty_sum(hg):
    """K = 0: the bias alone."""
    case(hg, 5, 70, 0, F16, "silu", R=True, save="16")
    case(hg, 5, 70, 0, BF16, "none", bias=False)


def test_large_tiles(hg):
    """Sizes that take the large tiles, ragged and with a partial last stage."""
    case(hg, 1000, 4100, 200, BF16, "gelu", R=True, save="8")
    case(hg, 4100, 4096, 72, F16, "silu", save="16")
    case(hg, 4133, 4001, 130, BF16, "relu", R=True, out=F32)


def test_limits(hg):
    """Sums past the type's range, infinities and NaN in single rows: they stay in their rows, and the activations
    take their limits."""
    M, N, K = 6, 40, 64
    X, W = torch.zeros(M, K), torch.zeros(N, K)
    X[0, 0], X[1, 0], X[2, 1], X[3, 2] = 60000.0, -60000.0, float("inf"), float("nan")
    W[:, 0], W[:, 1] = 4.0, 1.0
    for name in ref.ACTS:
        Y = torch.empty(M, N, dtype=F32, device=DEV)
        Z = hg.checkpoint8_empty(M, N, DEV)
        hg.linear(X.to(F16).to(DEV), W.to(F16).to(DEV), Y, act=act_of(hg, name), Z=Z)
        y = Y.cpu()
        low = -240000.0 if name == "none" else 0.0
        assert torch.allclose(y[0], torch.full((N,), 240000.0), rtol=2e-6) and torch.allclose(y[1], torch.full((N,), low)), name
        assert (y[2] == float("inf")).all() and y[3].isnan().all() and (y[4:] == 0).all()
        v = ref.values8(*Z)
        assert (v[0] == 240 * 256).all() and (v[1] == -240 * 256).all()
        assert v[2].isnan().all() and v[3].isnan().all() and (v[4:] == 0).all()
        X2 = X.clone()
        X2[2, 1] = float("-inf")
        hg.linear(X2.to(F16).to(DEV), W.to(F16).to(DEV), Y, act=act_of(hg, name))
        assert (Y.cpu()[2] == (float("-inf") if name == "none" else 0.0)).all(), name


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (40, 48, 16384), (300, 512, 264)])
def test_same_bits_every_time(hg, M, N, K):
    X, W = torch.randn(M, K, device=DEV).to(BF16), torch.randn(N, K, device=DEV).to(BF16)
    outs = [hg.linear(X, W, torch.empty(M, N, dtype=F32, device=DEV)).clone() for _ in range(4)]
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (33, 300, 4096), (300, 512, 129)])
def test_captured_and_replayed(hg, M, N, K):
    """On a stream of its own, captured once and replayed with other inputs between eager calls."""
    X, W = torch.empty(M, K, dtype=F16, device=DEV), torch.randn(N, K, device=DEV).to(F16)
    Y, Z = torch.empty(M, N, dtype=F16, device=DEV), torch.empty(M, N, dtype=F16, device=DEV)
    X.normal_()
    work = hg.linear_workspace(X, W)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        hg.linear(X, W, Y, act=hg.ACT_SILU, Z=Z, work=work)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        hg.linear(X, W, Y, act=hg.ACT_SILU, Z=Z, work=work)
    for seed in range(4):
        X.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(F16))
        graph.replay()
        torch.cuda.synchronize()
        got, gotz = Y.clone(), Z.clone()
        want, wantz = torch.empty_like(Y), torch.empty_like(Z)
        hg.linear(X, W, want, act=hg.ACT_SILU, Z=wantz)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(gotz, wantz), seed


def test_two_streams_with_their_own_workspaces(hg):
    M, N, K = 40, 96, 8192
    ins = [(torch.randn(M, K, device=DEV).to(F16), torch.randn(N, K, device=DEV).to(F16)) for _ in range(2)]
    want = [hg.linear(x, w, torch.empty(M, N, dtype=F32, device=DEV)).clone() for x, w in ins]
    torch.cuda.synchronize()
    outs, streams = [[], []], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(8):
        for i, (x, w) in enumerate(ins):
            with torch.cuda.stream(streams[i]):
                outs[i].append(hg.linear(x, w, torch.empty(M, N, dtype=F32, device=DEV)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in outs[i])


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (5, 40, 72), (100, 72, 17), (300, 256, 264)])
def test_columns_of_one_array(hg, M, N, K):
    """X, Y and Z side by side in one array, as slices of one tensor: the same bits as apart, nothing else written."""
    g = torch.Generator().manual_seed(M)
    big = torch.randn(M, K + 2 * N + 24, generator=g).to(BF16).to(DEV)
    W = torch.randn(N, K, generator=g).to(BF16).to(DEV)
    X, Y, Z = big[:, 8:8 + K], big[:, 8 + K:8 + K + N], big[:, 16 + K + N:16 + K + 2 * N]
    y, z = torch.empty(M, N, dtype=BF16, device=DEV), torch.empty(M, N, dtype=BF16, device=DEV)
    want = big.clone()
    hg.linear(X.contiguous(), W, y, act=act_of(hg, "silu"), Z=z)
    hg.linear(X, W, Y, act=act_of(hg, "silu"), Z=Z)
    want[:, 8 + K:8 + K + N] = y
    want[:, 16 + K + N:16 + K + 2 * N] = z
    assert torch.equal(big.view(torch.int16), want.view(torch.int16))


def test_row_of_a_wide_array(hg):
    """One row whose stride is past the largest leading dimension: a stride that no second row uses."""
    X = torch.ones(1, 64, dtype=F16, device=DEV).as_strided((1, 64), (1 << 40, 1))
    Y = torch.empty(1, 32, dtype=F16, device=DEV)
    hg.linear(X, torch.ones(32, 64, dtype=F16, device=DEV), Y)
    assert (Y == 64).all()


def test_an_error_that_another_call_left_is_not_reported(hg):
    """An earlier HIP call's error stays with it: the launches' own status is what counts."""
    hip = ctypes.CDLL(hg.LIB_PATH)                        # the runtime that the library is linked to
    X = torch.ones(4, 64, dtype=F16, device=DEV)
    W, Y = torch.ones(64, 64, dtype=F16, device=DEV), torch.empty(4, 64, dtype=F16, device=DEV)
    dW, pair = torch.empty_like(W), hg.checkpoint8_empty(4, 64)
    work = hg.linear_grad_workspace(Y, W, X)
    for call in (lambda: hg.linear(X, W, Y), lambda: hg.checkpoint8_write(X, *pair),
                 lambda: hg.linear_grad(Y, W, X, dW=dW, work=work)):
        assert hip.hipSetDevice(9999) != 0
        call()
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert (Y == 64).all() and (dW == 256).all()


def test_binding_refusals(hg):
    e = lambda m, n, t=F16: torch.zeros(m, n, dtype=t, device=DEV)  # noqa: E731
    X, W, Y = e(4, 16), e(8, 16), e(4, 8)
    for bad in (dict(X=e(4, 15)), dict(W=e(8, 16, BF16)), dict(Y=e(4, 9)), dict(bias=e(1, 8)[0]), dict(residual=e(4, 8, F32)),
                dict(residual=e(5, 8)), dict(Z=e(4, 8, F32)), dict(Z=(e(4, 8, torch.uint8), e(4, 2, torch.uint8))),
                dict(Z=7), dict(X=X[:1].expand(4, 16)), dict(X=e(16, 4).t()), dict(work=torch.zeros(4))):
        kw = dict(X=X, W=W, Y=Y) | bad
        with pytest.raises((TypeError, ValueError)):
            hg.linear(kw.pop("X"), kw.pop("W"), kw.pop("Y"), **kw)
    with pytest.raises(hg.HgError):
        hg.linear(X, W, Y, act=11)
    with pytest.raises(hg.HgError):
        hg.linear(X, W, X[:, :8])
    with pytest.raises(hg.HgError):
        hg.linear(e(100, 8200), e(64, 8200), e(100, 64), work=e(1, 1, torch.uint8))
