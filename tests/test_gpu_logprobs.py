"""hg_logprobs and hg_logprobs_grad against 64 bits.

Bounds.  u = 2^-24, D_j = scale·(x_j - x*).  The kernels form x_j - x*, multiply it
by scale·log2(e) (itself rounded) and take 2^: an exponent off by 3u·|D_j| and an
exponential off by 2u of itself, twice where parts are joined: each term of S is
off by (6·|D_j| + 8)u, and a sum of at most 64 in a lane, 64 lanes and 64 + 4 parts
by 150u more.  So S is off by rs = u·(6·Σ|D|p + 160) of itself; log S by rs +
2u·(1 + |log S|); log p = D - log S by that and 3u·(|D| + |log p|).  Σ D·e^D / S is
off by u·Σ p·|D|·(6·|D| + 170) + rs·Σ p·|D|, the entropy by that, log S and 3u of
either.  The gradient's exponent is off by e = u·(4·|D| + 4·|log S| + 3) + the
statistics' error, its p by that + 2u, and its terms by 8u of their magnitudes.
"""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24
INF = float("inf")


def logits(M, V, t, seed=0, spread=3.0, pad=0, shift=0):
    """(the logits on the CPU, the same on the device in rows of V + pad, `shift` elements past an aligned address)"""
    g = torch.Generator().manual_seed(seed * 1000003 + M * 7919 + V)
    x = (spread * torch.randn(M, V, generator=g)).to(t)
    return x, place(x, pad, shift)


def place(x, pad=0, shift=0):
    """In rows of V + pad with NaN around them."""
    M, V = x.shape
    buf = torch.full((M * (V + pad) + shift + 16,), float("nan"), dtype=x.dtype, device=DEV)
    v = buf[shift:shift + M * (V + pad)].view(M, V + pad)[:, :V]
    v.copy_(x)
    return v


def expected(x, scale):
    """{name: value} and {name: bound} of everything but the tokens', in 64 bits."""
    x = x.double()
    top = torch.where(x.isnan(), -INF, x).amax(1, keepdim=True)
    d = (x - torch.where(top == -INF, 0.0, top)) * scale
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    logs = torch.log(s)
    zero = lambda v: torch.where(e == 0, 0.0, v)  # noqa: E731
    p, ad = e / s, zero(d.abs())
    dp = (ad * p).sum(1, keepdim=True)
    rs = U * (6 * dp + 160)
    el = rs + 2 * U * (1 + logs.abs())
    entropy = logs - zero(d * p).sum(1, keepdim=True)
    eh = el + U * (p * ad * (6 * ad + 170)).sum(1, keepdim=True) + rs * dp + 3 * U * (logs.abs() + dp)
    nothing = s == 0
    logp = torch.where(nothing, -INF, d - logs)
    return dict(top=top, logs=logs, entropy=torch.where(nothing, 0.0, entropy), logp=logp, p=p, d=d), \
        dict(logs=el, entropy=eh, logp=el + 3 * U * (d.abs() + logp.abs()))


def close(got, want, bound, what):
    got = got.cpu().double()
    want = torch.where(want.abs() > torch.finfo(F32).max, want.sign() * INF, want)       # past fp32's range
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {float(got[i])!r}, expected "
                             f"{float(want[i])!r} within {float(bound.expand_as(want)[i])!r}")


def order(x, k):
    """The k largest's numbers, of equal ones the lower first, NaN as -inf."""
    return torch.where(x.isnan(), -INF, x.double()).sort(dim=1, descending=True, stable=True).indices[:, :k]


def run(hg, x, dev, tokens, k=0, scale=1.0, work=None):
    M, V = x.shape
    out = lambda *s, t=F32: torch.full(s, 55, dtype=t, device=DEV)  # noqa: E731
    logp, entropy, stats = out(M), out(M), out(M, 2)
    top = (out(M, k, t=torch.int64), out(M, k)) if k else None
    hg.logprobs(dev, tokens.to(DEV), logp=logp, entropy=entropy, stats=stats, top=top, scale=scale, work=work)
    return logp, entropy, stats, top


def check(hg, x, dev, tokens, k=0, scale=1.0):
    M, V = x.shape
    print(f"[logprobs] M={M} V={V} {x.dtype} k={k} scale={scale} ld={dev.stride(0)}", flush=True)
    logp, entropy, stats, top = run(hg, x, dev, tokens, k, scale)
    torch.cuda.synchronize()
    v, b = expected(x, scale)
    at = tokens.clamp(0, V - 1)[:, None]
    there = tokens[:, None] == at
    pick = lambda m, none: torch.where(there, m.gather(1, at), none)[:, 0]  # noqa: E731
    close(logp, pick(v["logp"], 0.0), pick(b["logp"], 0.0), "logp")
    close(entropy, v["entropy"][:, 0], b["entropy"][:, 0], "entropy")
    close(stats[:, 0], v["top"][:, 0], torch.zeros(M), "largest")
    close(stats[:, 1], v["logs"][:, 0], b["logs"][:, 0], "log of the sum")
    if k:
        ids = order(x, k)
        assert torch.equal(top[0].cpu(), ids)
        close(top[1], v["logp"].gather(1, ids), b["logp"].gather(1, ids), "top")
    return v, b, stats, entropy


def some_tokens(M, V, seed=3):
    g = torch.Generator().manual_seed(seed + M)
    t = torch.randint(0, V, (M,), generator=g)
    if M > 2:
        t[1], t[2] = -1, V
    return t


# one part and many, rows at odd places, one group and less
@pytest.mark.parametrize("t", [F16, BF16, F32])
@pytest.mark.parametrize("M,V,k,pad,shift", [
    (1, 1, 1, 0, 0), (3, 2, 2, 0, 1), (5, 7, 7, 0, 0), (5, 8, 3, 0, 3), (4, 9, 9, 1, 7), (9, 100, 32, 0, 0), (33, 1000, 5, 0, 0),
    (7, 2041, 20, 0, 0), (7, 2048, 20, 0, 5), (3, 2049, 32, 3, 0), (2, 5001, 1, 0, 0), (600, 4097, 8, 0, 0),
    (1, 50264, 20, 0, 0), (1, 131072, 32, 0, 0), (1100, 20001, 6, 0, 0), (513, 33000, 32, 0, 2), (2, 1 << 20, 32, 0, 1),
    (600, 300, 32, 0, 0), (1030, 16391, 4, 0, 0),
])
def test_forward(hg, t, M, V, k, pad, shift):
    x, dev = logits(M, V, t, pad=pad, shift=shift)
    check(hg, x, dev, some_tokens(M, V), k)


@pytest.mark.parametrize("scale", [0.25, 1.3, 4.0])
@pytest.mark.parametrize("M,V", [(5, 777), (3, 30000)])
def test_scale(hg, M, V, scale):
    x, dev = logits(M, V, BF16, pad=1)
    check(hg, x, dev, some_tokens(M, V), 12, scale)


@pytest.mark.parametrize("t", [F16, BF16, F32])
@pytest.mark.parametrize("V,k", [(300, 32), (9000, 17), (40000, 32)])
def test_equal_logits(hg, t, V, k):
    """All alike, two values, a staircase, zeros of both signs: the lower number first."""
    g = torch.Generator().manual_seed(V)
    n = torch.arange(V)
    rows = [torch.ones(V), (torch.rand(V, generator=g) < 0.01).float(), torch.full((V,), -INF), (n // 64).float() % 7,
            torch.where(n % 2 == 0, 0.0, -0.0), n.float().flip(0), n.float() / V, torch.where(n % 8 == 7, 1.0, -2.0),
            torch.where(n < V - 3, -INF, 1.0), torch.where(n % 2048 == 5, 3.0, -1.0)]
    x = torch.stack(rows).to(t)
    check(hg, x, place(x), torch.arange(len(rows)), k)


@pytest.mark.parametrize("t", [F16, BF16, F32])
@pytest.mark.parametrize("V,pad", [(5, 1), (1000, 0), (30001, 0)])
def test_masks_infinities_and_nan(hg, t, V, pad):
    """Rows whose mask leaves nothing, one token, all but one; the type's lowest value as a mask; its largest; +inf; NaN."""
    low = torch.finfo(t).min
    x, _ = logits(14, V, t)
    x[0] = -INF
    x[1] = -INF
    x[1, V - 1] = 2.0
    x[2, 0] = -INF
    x[3] = low
    x[4] = low
    x[4, 1] = 1.0
    x[5, 2] = torch.finfo(t).max
    x[6] = torch.finfo(t).max
    x[7, 3] = INF
    x[8, 4] = float("nan")
    x[9] = float("nan")
    x[10] = -INF
    x[10, 2] = float("nan")
    x[11, 1:] = low
    x[11, 0] = torch.finfo(t).max
    x[12] = -x[12].abs() - 100
    tokens = torch.tensor([0, V - 1, 0, 1, 1, 2, 0, 3, 0, 0, 2, 1, 3, -7])
    check(hg, x, place(x, pad), tokens, min(V, 8))


@pytest.mark.parametrize("t", [F16, BF16, F32])
@pytest.mark.parametrize("order_of", ["up", "down", "ends"])
def test_candidates_in_few_lanes(hg, t, order_of):
    """The largest logits next to each other, and eight lanes' worth of large ones: as many candidates as there can be."""
    V, k = 16384 * 2, 32
    n = torch.arange(V)
    x = {"up": n, "down": V - n, "ends": (n % 2048 < 64) * 1000 + (n * 37) % 61}[order_of].float() / 100
    if t != F32:
        x = x.to(t)
    x = x.to(t).expand(600, V).clone()
    check(hg, x, place(x), some_tokens(600, V), k)


def test_parts_of_a_call(hg):
    """Every output alone gives what all together do."""
    x, dev = logits(6, 9000, BF16)
    tokens = some_tokens(6, 9000).to(DEV)
    logp, entropy, stats, top = run(hg, x, dev, tokens.cpu(), 5)
    new = lambda v: torch.empty_like(v)  # noqa: E731
    assert torch.equal(hg.logprobs(dev, tokens, logp=new(logp))[0], logp)
    assert torch.equal(hg.logprobs(dev, entropy=new(entropy))[1], entropy)
    assert torch.equal(hg.logprobs(dev, stats=new(stats))[2], stats)
    assert torch.equal(hg.logprobs(dev, top=(new(top[0]), None))[3][0], top[0])
    assert torch.equal(hg.logprobs(dev, top=(None, new(top[1])))[3][1], top[1])
    hg.logprobs(dev)


def gradient(x, tokens, scale, dl, dh, v, b):
    """(the gradient, its bound before the last rounding)"""
    M, V = x.shape
    at = tokens.clamp(0, V - 1)[:, None]
    there = (tokens[:, None] == at)
    dl = torch.where(there, dl.double()[:, None], 0.0) if dl is not None else torch.zeros(M, 1).double()
    dh = dh.double()[:, None] if dh is not None else torch.zeros(M, 1).double()
    live = v["p"] > 0
    z = lambda m: torch.where(live, m, 0.0)  # noqa: E731
    p, lp, h = z(v["p"]), z(v["logp"]), v["entropy"]
    e = z(U * (4 * v["d"].abs() + 4 * v["logs"].abs() + 3) + b["logs"])
    one = torch.zeros(M, V).double().scatter_(1, at, there.double())
    g = scale * (dl * one - dl * p - dh * p * (lp + h))
    eh = b["entropy"] if dh.any() else torch.zeros(M, 1).double()
    size = dl.abs() * (p + one) + dh.abs() * p * (lp.abs() + h.abs())
    err = dl.abs() * p * (e + 2 * U) + dh.abs() * p * ((e + 2 * U) * (lp.abs() + h.abs()) + e + eh) + 8 * U * size
    nothing = v["logs"] == -INF
    return torch.where(nothing, 0.0, g), scale * torch.where(nothing, 0.0, err)


@pytest.mark.parametrize("t", [F16, BF16, F32])
@pytest.mark.parametrize("M,V,pad,shift,dpad,dshift", [
    (1, 1, 0, 0, 0, 0), (3, 2, 0, 1, 1, 0), (5, 9, 1, 3, 0, 7), (33, 1000, 0, 0, 0, 0), (7, 8192, 0, 0, 8, 0),
    (2, 8193, 0, 0, 0, 0), (20, 50264, 0, 0, 0, 3), (300, 777, 0, 0, 3, 0),
])
@pytest.mark.parametrize("which", ["both", "logp", "entropy"])
def test_gradient(hg, t, M, V, pad, shift, dpad, dshift, which):
    print(f"[logprobs_grad] M={M} V={V} {t} pad={pad} shift={shift} dpad={dpad} {which}", flush=True)
    x, dev = logits(M, V, t, pad=pad, shift=shift)
    tokens, scale = some_tokens(M, V), 0.8
    v, b, stats, entropy = check(hg, x, dev, tokens, 0, scale)
    g = torch.Generator().manual_seed(V)
    dl = torch.randn(M, generator=g) if which != "entropy" else None
    dh = torch.randn(M, generator=g) if which != "logp" else None
    buf = torch.full((M + 2, V + dpad + dshift), -77.0, dtype=t, device=DEV)
    dX = buf[1:M + 1, dshift:V + dshift]
    got = hg.logprobs_grad(dev, tokens.to(DEV), stats, dX, dlogp=None if dl is None else dl.to(DEV),
                           dentropy=None if dh is None else dh.to(DEV), entropy=entropy, scale=scale)
    assert got is dX
    torch.cuda.synchronize()
    ref.check(dX, *gradient(x, tokens, scale, dl, dh, v, b), "dX")
    buf[1:M + 1, dshift:V + dshift] = -77
    assert (buf == -77).all()


@pytest.mark.parametrize("t", [F16, BF16, F32])
@pytest.mark.parametrize("V", [17, 1000, 20001])
def test_gradient_in_place_and_masked(hg, t, V):
    """In place at odd rows; rows whose mask leaves nothing give zeros, as masked tokens do; NaN stays in its row."""
    x, _ = logits(40, V, t)
    x[:, V // 2:V // 2 + 3] = -INF
    x[3] = -INF
    x[5, 1] = float("nan")
    x[6] = torch.finfo(t).min
    x[7, 4] = 60.0
    tokens = some_tokens(40, V)
    tokens[7] = 4
    tokens[8] = V // 2
    dev = place(x, 0, 3)
    v, b, stats, entropy = check(hg, x, dev, tokens)
    g = torch.Generator().manual_seed(V)
    dl, dh = torch.randn(40, generator=g), torch.randn(40, generator=g)
    hg.logprobs_grad(dev, tokens.to(DEV), stats, dev, dlogp=dl.to(DEV), dentropy=dh.to(DEV), entropy=entropy)
    want, err = gradient(x, tokens, 1.0, dl, dh, v, b)
    rows = [i for i in range(40) if i != 5]
    ref.check(dev[rows], want[rows], err[rows], "dX")
    assert dev[5].isnan().any() and (dev[3] == 0).all()


def test_gradient_against_differences(hg):
    """fp32 logits: the gradient is the change of dl·log p + dh·H along a direction."""
    M, V = 6, 300
    x, dev = logits(M, V, F32, spread=1.5)
    tokens = some_tokens(M, V)
    g = torch.Generator().manual_seed(1)
    dl, dh, way = torch.randn(M, generator=g), torch.randn(M, generator=g), torch.randn(M, V, generator=g)
    _, entropy, stats, _ = run(hg, x, dev, tokens)
    dX = hg.logprobs_grad(dev, tokens.to(DEV), stats, torch.empty_like(dev), dlogp=dl.to(DEV), dentropy=dh.to(DEV),
                          entropy=entropy).cpu().double()

    def value(at):
        v, _ = expected(at, 1.0)
        there = (tokens >= 0) & (tokens < V)
        logp = torch.where(there, v["logp"].gather(1, tokens.clamp(0, V - 1)[:, None])[:, 0], 0.0)
        return dl.double() * logp + dh.double() * v["entropy"][:, 0]

    step = 1e-4
    change = (value(x.double() + step * way) - value(x.double() - step * way)) / (2 * step)
    # third derivatives of log p and H are below 30 per direction cubed (|way|³ < 100): step² · 500; sums of fp32 results
    lim = step ** 2 * 500 + 300 * 2.0 ** -20
    assert ((dX * way).sum(1) - change).abs().max() < lim


def test_offsets_past_32_bits(hg):
    """The last rows of logits of 2^32 bytes and more."""
    M, V = 70000, 32768
    x = torch.zeros(M, V, dtype=BF16, device=DEV)
    tail, _ = logits(3, V, BF16)
    x[-3:] = tail.to(DEV)
    tokens = torch.zeros(M, dtype=torch.int64)
    tokens[-3:] = torch.tensor([5, 6, V - 1])
    tokens = tokens.to(DEV)
    logp, stats = torch.empty(M, device=DEV), torch.empty(M, 2, device=DEV)
    ids = torch.empty(M, 4, dtype=torch.int64, device=DEV)
    hg.logprobs(x, tokens, logp=logp, stats=stats, top=(ids, None))
    v, b = expected(tail, 1.0)
    at = tokens[-3:].cpu()[:, None]
    close(logp[-3:], v["logp"].gather(1, at)[:, 0], b["logp"].gather(1, at)[:, 0], "logp")
    assert torch.equal(ids[-3:].cpu(), order(tail, 4)) and torch.equal(ids[:1].cpu(), torch.arange(4)[None])
    hg.logprobs_grad(x, tokens, stats, x, dlogp=torch.ones(M, device=DEV))
    want, err = gradient(tail, tokens[-3:].cpu(), 1.0, torch.ones(3), None, v, b)
    ref.check(x[-3:], want, err, "dX")


@pytest.mark.parametrize("M,V", [(2, 777), (4, 40000)])
def test_graph(hg, M, V):
    x, dev = logits(M, V, BF16)
    tokens = some_tokens(M, V).to(DEV)
    dl, dX = torch.ones(M, device=DEV), torch.empty_like(dev)
    logp, entropy, stats = (torch.empty(*s, device=DEV) for s in ((M,), (M,), (M, 2)))
    top = (torch.empty(M, 5, dtype=torch.int64, device=DEV), torch.empty(M, 5, device=DEV))
    work = hg.logprobs_workspace(dev, 5)

    def both(to):
        hg.logprobs(dev, tokens, logp=logp, entropy=entropy, stats=stats, top=top, work=work)
        hg.logprobs_grad(dev, tokens, stats, to, dlogp=dl)

    with torch.cuda.stream(torch.cuda.Stream()):
        both(dX)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(dX)
    for i in range(4):
        dev.copy_(3 * torch.randn(M, V, device=DEV))
        tokens.copy_(torch.randint(0, V, (M,), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (logp, entropy, stats, *top, dX)]
        both(dX)
        for a, b in zip(got, (logp, entropy, stats, *top, dX)):
            assert torch.equal(a, b), i


def test_two_calls_at_once(hg):
    """On two streams, each with its own workspace."""
    xs = [logits(3, 60000, BF16, seed=s) for s in range(2)]
    tokens = some_tokens(3, 60000)
    want = [run(hg, x, dev, tokens, 9) for x, dev in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for (x, dev), stream in zip(xs, streams):
            with torch.cuda.stream(stream):
                got.append(run(hg, x, dev, tokens, 9))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1]) and torch.equal(g[3][0], w[3][0])


def test_more_rows_than_a_launch_has_workgroups(hg):
    """Workgroups that go on to further rows, of one part and of several."""
    for M, V, k in (((1 << 22) + 77, 9, 3), ((1 << 20) + 7, 4100, 1)):
        g = torch.Generator(device=DEV).manual_seed(M)
        x = (3 * torch.randn(M, V, generator=g, device=DEV)).to(BF16)
        tokens = torch.randint(0, V, (M,), generator=g, device=DEV)
        logp, stats = torch.full((M,), 9.0, device=DEV), torch.empty(M, 2, device=DEV)
        ids = torch.full((M, k), -5, dtype=torch.int64, device=DEV)
        hg.logprobs(x, tokens, logp=logp, stats=stats, top=(ids, None))
        rows = torch.cat((torch.arange(50), torch.randint(0, M, (200,), generator=torch.Generator().manual_seed(1)),
                          torch.arange(M - 100, M)))
        some, tok = x[rows.to(DEV)].cpu(), tokens[rows.to(DEV)].cpu()
        v, b = expected(some, 1.0)
        close(logp[rows.to(DEV)], v["logp"].gather(1, tok[:, None])[:, 0], b["logp"].gather(1, tok[:, None])[:, 0], "logp")
        assert torch.equal(ids[rows.to(DEV)].cpu(), order(some, k))
        assert (logp <= 1e-4).all() and (ids >= 0).all()                     # every row was written
        hg.logprobs_grad(x, tokens, stats, x, dlogp=torch.ones(M, device=DEV))
        want, err = gradient(some, tok, 1.0, torch.ones(len(rows)), None, v, b)
        ref.check(x[rows.to(DEV)], want, err, "dX")
