"""hg_linear_grad against 64 bits (linear_ref.py: formulas and bounds) and
against differences of the layer itself."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def act_of(hg, name):
    return getattr(hg, "ACT_" + name.upper())


def strided(x, pad, shift=0):
    M, N = x.shape
    buf = torch.full((M * (N + pad) + shift + 16,), float("nan"), dtype=x.dtype, device=DEV)
    v = buf[shift:shift + M * (N + pad)].view(M, N + pad)[:, :N]
    v.copy_(x)
    return v


def room(M, N, t, pad, fill=None):
    buf = torch.full((M + 2, N + pad), -77.0, dtype=t, device=DEV)
    out = buf[1:M + 1, :N]
    if fill is not None:
        out.copy_(fill)

    def untouched():
        assert (buf[0] == -77).all() and (buf[M + 1] == -77).all() and (buf[:, N:] == -77).all()
    return out, untouched


def case(hg, M, N, K, t=F16, name="silu", dw=None, accumulate=False, x8=False, z8=False, pad=0, shift=0, want="xwb",
         integers=False, seed=0):
    print(f"[grad] M={M} N={N} K={K} {t} {name} dw={dw} acc={accumulate} x8={x8} z8={z8} pad={pad} shift={shift} "
          f"{want}", flush=True)
    g = torch.Generator().manual_seed(seed * 1000003 + M * 7919 + N * 31 + K)
    rnd = (lambda *s: torch.randint(-2, 3, s, generator=g).to(t)) if integers else \
        (lambda *s: torch.randn(*s, generator=g).to(t))
    dY, W, X, Z = rnd(M, N), rnd(N, K), rnd(M, K), rnd(M, N)
    dw = dw or t
    Xd, Zd = strided(X, pad, shift), strided(Z, pad, shift)
    if x8:
        Xd = hg.checkpoint8_write(Xd, *hg.checkpoint8_empty(M, K, DEV))
        X = ref.codes8(X)[0]
    if z8:
        Zd = hg.checkpoint8_write(Zd, *hg.checkpoint8_empty(M, N, DEV))
        Z = ref.codes8(Z)[0]
    dYd, Wd = strided(dY, pad, shift), strided(W, pad, shift)
    w0 = torch.randint(-4, 5, (N, K), generator=g).to(dw) if accumulate else None
    b0 = torch.randint(-4, 5, (N,), generator=g).float() if accumulate else None
    dX, ax = room(M, K, t, pad)
    dW, aw = room(N, K, dw, pad, w0)
    db = torch.full((N,), 5.0, device=DEV) if b0 is None else b0.to(DEV)
    need = hg.linear_grad_workspace_size(dYd, Wd if "x" in want else None, Xd if "w" in want else None)
    work = torch.full((need // 2 + 8,), float("nan"), dtype=F16, device=DEV)
    hg.linear_grad(dYd, Wd if "x" in want else None, Xd if "w" in want else None, Z=Zd if name != "none" else None,
                   act=act_of(hg, name), dX=dX if "x" in want else None, dW=dW if "w" in want else None,
                   dbias=db if "b" in want else None, accumulate=accumulate, work=work)
    torch.cuda.synchronize()
    ax()
    aw()
    r = ref.grads(dY, W, X, Z, name)
    for key, out, base in (("dX", dX, None), ("dW", dW, w0), ("dbias", db, b0)):
        v, e = r[key]
        if key[1].lower() not in want:
            assert (out.cpu() == (-77.0 if base is None else base) if key != "dbias" else
                    (out.cpu() == (5.0 if base is None else base))).all(), key
            continue
        if base is not None:
            v = v + base.double()
            e = e + ref.U32 * (v.abs() + e)
        if integers:
            assert torch.equal(out.cpu().double(), v.to(out.dtype).double()), key
        ref.check(out, v, e, key)


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 1000, 72), (2, 33, 40), (3, 257, 130), (7, 8, 1000), (16, 96, 136), (17, 65, 72),
          (33, 100, 64), (64, 64, 64), (65, 63, 65), (100, 300, 520), (128, 256, 1024), (129, 129, 129), (250, 511, 333),
          (300, 130, 136), (1000, 40, 48), (4097, 32, 24), (2051, 64, 136)]


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(hg, M, N, K, t):
    case(hg, M, N, K, t)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_integers_are_exact(hg, M, N, K):
    case(hg, M, N, K, F16, "relu", dw=F32, integers=True)
    case(hg, M, N, K, BF16, "none", dw=F32, integers=True, pad=3)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("x8,z8", [(False, False), (True, False), (False, True), (True, True)])
def test_activations_and_checkpoints(hg, name, x8, z8):
    case(hg, 70, 130, 96, BF16, name, x8=x8, z8=z8)
    case(hg, 37, 77, 100, F16, name, dw=F32, x8=x8, z8=z8, pad=3)
    case(hg, 300, 264, 320, F16, name, x8=x8, z8=z8)


@pytest.mark.parametrize("dw", [F16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (70, 65, 33), (300, 512, 256), (5000, 64, 72)])
def test_accumulate(hg, M, N, K, dw):
    case(hg, M, N, K, F16, "gelu", dw=dw, accumulate=True)
    case(hg, M, N, K, F16, "none", dw=dw, accumulate=True, integers=True, pad=8)


@pytest.mark.parametrize("want", ["x", "w", "b", "xw", "xb", "wb"])
def test_only_what_is_wanted(hg, want):
    case(hg, 70, 130, 96, F16, "silu", want=want)
    case(hg, 70, 136, 96, BF16, "none", want=want)
    case(hg, 201, 131, 97, BF16, "gelu_tanh", want=want)


@pytest.mark.parametrize("M,N,K", [(128, 1024, 2048), (1024, 512, 256), (300, 130, 2000), (64, 4096, 128)])
def test_one_workspace_for_any_gradients(hg, M, N, K):
    """The size for both operands is enough whichever gradients are wanted."""
    dY, W, X, Z = (torch.randn(s, device=DEV).to(F16) for s in ((M, N), (N, K), (M, K), (M, N)))
    work = hg.linear_grad_workspace(dY, W, X)
    kw = dict(Z=Z, act=hg.ACT_SILU, work=work)
    for one in (dict(dX=torch.empty_like(X)), dict(dW=torch.empty_like(W)), dict(dbias=torch.empty(N, device=DEV)),
                dict(dX=torch.empty_like(X), dW=torch.empty_like(W))):
        hg.linear_grad(dY, W, X, **one, **kw)
        for key, out in one.items():
            ref.check(out, *ref.grads(dY.cpu(), W.cpu(), X.cpu(), Z.cpu(), "silu")[key], key)


@pytest.mark.parametrize("pad,shift", [(0, 1), (0, 8), (1, 0), (8, 0), (64, 4), (5, 3)])
def test_strides_and_alignment(hg, pad, shift):
    case(hg, 75, 136, 200, F16, "silu", pad=pad, shift=shift)
    case(hg, 75, 136, 200, BF16, "none", pad=pad, shift=shift)
    case(hg, 130, 77, 35, F16, "relu", pad=pad, shift=shift, dw=F32)


def test_large_tiles(hg):
    case(hg, 4100, 4096, 72, BF16, "gelu_tanh")
    case(hg, 200, 4100, 4096, F16, "silu", x8=True, z8=True)
    case(hg, 4133, 130, 4001, BF16, "relu", dw=F32)


def test_empty(hg):
    e = lambda m, n, t=F16: torch.full((m, n), 3.0, dtype=t, device=DEV)  # noqa: E731
    dW, db = e(8, 16, F32), torch.full((8,), 3.0, device=DEV)
    hg.linear_grad(e(0, 8), e(8, 16), e(0, 16), Z=e(0, 8), act=hg.ACT_SILU, dX=e(0, 16), dW=dW, dbias=db,
                   accumulate=True)
    assert (dW == 3).all() and (db == 3).all()
    hg.linear_grad(e(0, 8), e(8, 16), e(0, 16), Z=e(0, 8), act=hg.ACT_SILU, dX=e(0, 16), dW=dW, dbias=db)
    assert (dW == 0).all() and (db == 0).all()
    dX = e(4, 16)
    hg.linear_grad(e(4, 0), e(0, 16), e(4, 16), dX=dX, dW=e(0, 16), dbias=torch.empty(0, device=DEV))
    assert (dX == 0).all()
    db = torch.full((8,), 3.0, device=DEV)
    hg.linear_grad(e(4, 8), e(8, 0), e(4, 0), dX=e(4, 0), dW=e(8, 0), dbias=db)
    assert (db == 12).all()


def test_limits(hg):
    """Slopes at ±inf are the limits, at NaN NaN; ReLU's zero slope drops an infinite dY."""
    inf, nan = float("inf"), float("nan")
    Z = torch.tensor([[inf, -inf, nan, 0.0, -1.0, 1.0, 30.0, -30.0]], dtype=F16, device=DEV)
    dY = torch.full((1, 8), 2.0, dtype=F16, device=DEV)
    for name in ref.ACTS[1:]:
        db = torch.empty(8, device=DEV)
        hg.linear_grad(dY, None, None, Z=Z, act=act_of(hg, name), dbias=db)
        v = db.cpu()
        assert v[0] == 2 and v[1] == 0 and v[2].isnan() and v[6] == 2 and abs(float(v[7])) < 1e-5, (name, v)
        assert v[3] == (0 if name == "relu" else 1)
    dY[0, 4] = inf
    hg.linear_grad(dY, None, None, Z=Z, act=hg.ACT_RELU, dbias=db)
    assert db[4] == 0


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("name", ref.ACTS[1:])
def test_slopes_of_every_value(hg, name, t):
    """act' of all 2^16 values of a type, from dbias of one row with dY = 1.  Roundings of the formula: the
    logistic's exponent is off by 2^-23 of itself (at most 2^-17 where e·s² is above 2^-40) and its factors by a few
    2^-23; z·phi(z) and z·w·e·s² stay below 1.2; Phi's own formula is off by 0.75e-7: 2^-19 together."""
    Z = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(1, -1).view(t)
    db = torch.empty(65536, device=DEV)
    hg.linear_grad(torch.ones(1, 65536, dtype=t, device=DEV), None, None, Z=Z.to(DEV), act=act_of(hg, name), dbias=db)
    z, got = Z[0].double(), db.cpu().double()
    fine = z.isfinite()
    want = ref.slope(z.clamp(-200, 200), name)          # constant beyond
    assert ((got - want).abs()[fine] <= 2.0 ** -19).all(), float((got - want).abs()[fine].max())
    assert got[z.isnan()].isnan().all()
    assert (got[z == float("inf")] == 1).all() and (got[z == float("-inf")] == 0).all()


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("name", ref.ACTS)
def test_activations_of_every_value(hg, name, t):
    """act of all 2^16 values of a type through linear with K = 1, X = 1: within 2^-20·|z| (linear_ref.py)."""
    W = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(-1, 1).view(t)
    Y = torch.empty(1, 65536, device=DEV)
    hg.linear(torch.ones(1, 1, dtype=t, device=DEV), W.to(DEV), Y, act=act_of(hg, name))
    z, got = W[:, 0].double(), Y[0].cpu().double()
    fine = z.isfinite()
    want = ref.act(z, name)
    if name != "none":
        want = torch.where(z < -100, 0.0, want)         # where 64 bits meet inf times zero
    assert ((got - want).abs()[fine] <= 2.0 ** -20 * z.abs()[fine] + 2.0 ** -149).all()
    assert got[z.isnan()].isnan().all()
    assert (got[z == float("inf")] == float("inf")).all()
    assert (got[z == float("-inf")] == (float("-inf") if name == "none" else 0)).all()


def test_padding_is_not_read(hg):
    """NaN behind the last column of every operand (strided() puts it there) reaches nothing: K and N no multiple of
    8 or 64, the last chunk and the last stage of every sum partial."""
    case(hg, 66, 70, 75, BF16, "silu", pad=5)
    case(hg, 66, 72, 80, BF16, "silu", pad=8)


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_against_differences(hg, name):
    """L(X, W, b) = Σ dY·act(X·Wᵀ + b): the gradients from a forward call's saved pre-activation against central
    differences of L along random directions, in 64 bits.  The difference's own error is h²/6·|L'''| with h = 1e-4
    and |act'''| <= 2; the gradients carry the bounds of grads() and the saved Z's rounding times |act''| <= 1."""
    M, N, K, t = 24, 40, 56, F16
    g = torch.Generator().manual_seed(5)
    X, W, dY = (torch.randn(s, generator=g).to(t) for s in ((M, K), (N, K), (M, N)))
    W = (W / K ** 0.5).to(t)
    b = torch.randn(N, generator=g)
    Y, Z = torch.empty(M, N, dtype=t, device=DEV), torch.empty(M, N, dtype=t, device=DEV)
    hg.linear(X.to(DEV), W.to(DEV), Y, bias=b.to(DEV), act=act_of(hg, name), Z=Z)
    dX, dW, db = torch.empty(M, K, dtype=t, device=DEV), torch.empty(N, K, dtype=F32, device=DEV), torch.empty(N, device=DEV)
    hg.linear_grad(dY.to(DEV), W.to(DEV), X.to(DEV), Z=Z, act=act_of(hg, name), dX=dX, dW=dW, dbias=db)
    z = Z.cpu().double()
    r = ref.grads(dY, W, X, Z.cpu(), name)
    dz = dY.double().abs() * ref.half(t) * (z.abs() + 2.0 ** -14)      # what Z's rounding does to dz
    more = {"dX": dz @ W.double().abs(), "dW": dz.t() @ X.double().abs(), "dbias": dz.sum(0)}
    loss = lambda x, w, c: float((dY.double() * ref.act(x @ w.t() + c, name)).sum())  # noqa: E731
    x, w, c, h = X.double(), W.double(), b.double(), 1e-4
    for key, out in (("dX", dX), ("dW", dW), ("dbias", db)):
        for _ in range(3):
            v = torch.randn(out.shape, generator=g, dtype=torch.float64)
            args = lambda s: (x + s * v if key == "dX" else x, w + s * v if key == "dW" else w,  # noqa: E731,B023
                              c + s * v if key == "dbias" else c)
            diff = (loss(*args(h)) - loss(*args(-h))) / (2 * h)
            got = float((out.cpu().double() * v).sum())
            move = (v @ w.t() if key == "dX" else x @ v.t() if key == "dW" else v.expand(M, N)).abs()
            lim = float(((r[key][1] + more[key] + ref.half(out.dtype) * out.cpu().double().abs() + 2.0 ** -25)
                         * v.abs()).sum()) + h * h / 6 * 2 * float((dY.double().abs() * move ** 3).sum()) + 1e-7
            assert abs(got - diff) <= lim, (key, got, diff, lim)


def test_a_step_with_8_bit_checkpoints(hg):
    """Forward, both checkpoints, backward, as a training loop calls them, captured and replayed as well; the
    gradients are those of the values that the checkpoints stand for."""
    M, N, K, t, name = 200, 300, 264, BF16, "gelu"
    g = torch.Generator().manual_seed(9)
    X, dY = torch.randn(M, K, generator=g).to(t).to(DEV), torch.randn(M, N, generator=g).to(t).to(DEV)
    W, b = (torch.randn(N, K, generator=g) / K ** 0.5).to(t).to(DEV), torch.randn(N, generator=g).to(DEV)
    X8, Z8 = hg.checkpoint8_empty(M, K, DEV), hg.checkpoint8_empty(M, N, DEV)
    Y, dX, dW, db = (torch.empty(s, dtype=u, device=DEV) for s, u in (((M, N), t), ((M, K), t), ((N, K), F32), ((N,), F32)))
    work, gwork = hg.linear_workspace(X, W), hg.linear_grad_workspace(dY, W, X8)

    def step():
        hg.checkpoint8_write(X, *X8)
        hg.linear(X, W, Y, bias=b, act=hg.ACT_GELU, residual=None, Z=Z8, work=work)
        hg.linear_grad(dY, W, X8, Z=Z8, act=hg.ACT_GELU, dX=dX, dW=dW, dbias=db, work=gwork)

    def right():
        torch.cuda.synchronize()
        y, z, ey, ez = ref.linear(X.cpu(), W.cpu(), b.cpu(), name)
        ref.check(Y, y, ey, "Y")
        r = ref.grads(dY.cpu(), W.cpu(), ref.values8(*X8), ref.values8(*Z8), name)
        for key, out in (("dX", dX), ("dW", dW), ("dbias", db)):
            ref.check(out, *r[key], key)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    right()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in range(3):
        X.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(t))
        for o in (Y, dX, dW, db):
            o.fill_(7.0)
        graph.replay()
        right()
        kept = [o.clone() for o in (Y, dX, dW, db)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, o) for a, o in zip(kept, (Y, dX, dW, db)))


def test_binding_refusals(hg):
    e = lambda m, n, t=F16: torch.zeros(m, n, dtype=t, device=DEV)  # noqa: E731
    ok = dict(dY=e(4, 8), W=e(8, 16), X=e(4, 16), Z=e(4, 8), act=hg.ACT_SILU, dX=e(4, 16), dW=e(8, 16))
    for bad in (dict(W=None), dict(X=None), dict(Z=None), dict(dX=e(4, 15)), dict(dW=e(7, 16)), dict(dbias=e(1, 8)),
                dict(W=e(9, 16)), dict(X=e(5, 16)), dict(Z=e(4, 9)), dict(dW=e(8, 16, BF16)), dict(dX=e(4, 16, F32)),
                dict(X=(e(4, 16, torch.uint8), e(4, 2, torch.uint8)))):
        kw = ok | bad
        with pytest.raises((TypeError, ValueError)):
            hg.linear_grad(kw.pop("dY"), kw.pop("W"), kw.pop("X"), **kw)
    with pytest.raises(hg.HgError):
        hg.linear_grad(**(ok | dict(dX=ok["X"])))
    with pytest.raises(hg.HgError):
        hg.linear_grad(**ok, work=e(1, 16, torch.uint8))
