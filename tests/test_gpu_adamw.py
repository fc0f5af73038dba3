"""hg_adamw against its definition.

The moments' fp32 products and sums are each rounded by themselves, so fp32
moments, and the codes and scales of 8-bit ones, are known to the bit: the
reference forms them in fp32 on the CPU and rounds at random by the same bits.

The weight, from these moments, is in 64 bits; bound: u = 2^-24.  1 - beta^t is
off by 5u of itself (its exponent by u, expm1 by 4u), its reciprocal and its
product with either moment by 7u, half of that in the root, the card's root and
reciprocal by 2u each (a step), the sum with eps and the quotient one rounding
each: under 17u; times lr and with decay·w four more roundings of either term, the
subtraction one of the result, and factors one of lr.
"""
import numpy as np
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24
LR, B1, B2, EPS, DECAY = 3e-3, 0.9, 0.999, 1e-8, 0.1


def mix(x):
    x = x ^ (x >> np.uint32(16))
    x = x * np.uint32(0x9E3779B9)
    x = x ^ (x >> np.uint32(15))
    x = x * np.uint32(0xB504F333)
    return x ^ (x >> np.uint32(16))


def bits(seed, t, place, first, n):
    """The random bits of elements first .. first + n - 1."""
    at = np.arange(first, first + n, dtype=np.uint64)
    key = np.zeros(n, np.uint32)
    for w in (place, t & 0xffffffff, t >> 32, seed & 0xffffffff, seed >> 32, (at >> np.uint64(32)).astype(np.uint32)):
        key = mix(key + np.asarray(w, np.uint32) + np.uint32(0x9E3779B9))
    return mix(at.astype(np.uint32) ^ key)


GRID = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()      # 0 .. 448


def rounded(x, r, keep):
    """(codes, scale bytes) of fp32 x: the scale by search, the two nearest codes from a table, the upper one with
    r + 1/2 of 2^16 against the distance."""
    n = len(x)
    pad = np.zeros(-(-n // 32) * 32, np.float32)
    pad[:n] = x
    blocks = pad.reshape(-1, 32)
    fine = np.isfinite(blocks)
    amax = np.abs(np.where(fine, blocks, 0)).max(1).astype(np.float64)
    e = np.full(len(blocks), -117)
    for _ in range(237):
        e = np.where((amax > 448 * np.exp2(e.astype(np.float64))) & (e < 120), e + 1, e)
    y = (np.abs(blocks.astype(np.float64)) * np.exp2(-e.astype(np.float64))[:, None]).reshape(-1)[:n]
    y = np.where(np.isfinite(y), np.minimum(y, np.where(e == 120, 240.0, 448.0).repeat(32)[:n]), 0)
    # near zero the kernel's sum with 2^-6 is an fp32 one
    y32 = y.astype(np.float32)
    y = np.where(y < 2.0 ** -6, (y32 + np.float32(2.0 ** -6)).astype(np.float64) - 2.0 ** -6, y)
    k = np.clip(np.searchsorted(GRID, y, side="right") - 1, 0, 125)
    # (what is below a 2^20-th of the distance between codes is cut off)
    part = np.floor((y - GRID[k]) / (GRID[k + 1] - GRID[k]) * 2.0 ** 20)
    code = k + (part + r.astype(np.float64) * 16 + 8 >= 2.0 ** 20)
    if keep:
        code = np.where((code == 0) & (y32 > 0), 1, code)
    sign = np.signbit(x)
    code = np.where(np.isfinite(x), code, 127)
    return (code + 128 * sign).astype(np.uint8), (e + 127).astype(np.uint8)


def values(codes, scales):
    c = codes.view(torch.float8_e4m3fn).float().numpy()
    return c * np.exp2(scales.numpy().astype(np.float32) - 127).repeat(32)[:len(c)]


def step_of(g, m, v, w, t, lr=LR, gs=None, b1=B1, b2=B2, eps=EPS, decay=DECAY):
    """(m, v in fp32, weight in 64 bits, its bound) of numpy fp32 arrays."""
    f = np.float32
    with np.errstate(all="ignore"):
        s = g if gs is None else g * f(gs)
        m = f(b1) * m + f(1 - b1) * s
        v = f(b2) * v + f(1 - b2) * (s * s)
        w, d = w.astype(np.float64), float(f(decay))
        q = (m.astype(np.float64) / (1 - b1 ** t)) / (np.sqrt(v.astype(np.float64) / (1 - b2 ** t)) + float(f(eps)))
        new = w - float(f(lr)) * (d * w + q)
        err = lr * 1.01 * U * (6 * np.abs(d * w) + 24 * np.abs(q)) + U * np.abs(new)
    return m, v, torch.from_numpy(new), torch.from_numpy(err)


class Buffers:
    """Tensors one after the other in one buffer of each kind, `gap` elements between them, which must stay as they are."""

    def __init__(self, sizes, t, bits, master, gap=0, gtype=None, seed=0, shift=0):
        g = torch.Generator().manual_seed(seed)
        self.sizes, self.t, self.bits = sizes, t, bits
        at, self.at, self.sat, blocks = shift, [], [], 0
        for n in sizes:
            self.at.append(at)
            self.sat.append(blocks)
            at += n + gap
            blocks += -(-n // 32) + (gap > 0)
        total = max(1, at)
        rand = lambda: torch.randn(total, generator=g)  # noqa: E731
        self.w = rand() if master else None
        self.p = (self.w if master else rand()).to(t)
        self.g = (0.1 * rand() * torch.exp(rand())).to(gtype or t)
        self.m = 0.1 * rand()
        self.v = 0.01 * rand().square()
        self.scales = []
        if bits == 8:
            half = np.full(total, 1 << 15)
            for name, keep in (("m", False), ("v", True)):
                codes, scales = torch.zeros(total, dtype=torch.uint8), torch.zeros(max(1, blocks), dtype=torch.uint8)
                for a, s, n in zip(self.at, self.sat, sizes):
                    c, e = rounded(getattr(self, name)[a:a + n].numpy(), half[:n], keep)
                    codes[a:a + n], scales[s:s + len(e)] = torch.from_numpy(c), torch.from_numpy(e)
                setattr(self, name, (codes, scales))
        self.dev = {k: (tuple(x.to(DEV) for x in v) if isinstance(v, tuple) else v.to(DEV) if v is not None else None)
                    for k, v in (("p", self.p), ("w", self.w), ("g", self.g), ("m", self.m), ("v", self.v))}

    def parts(self, kind):
        x = self.dev[kind]
        if x is None:
            return None
        if isinstance(x, tuple):
            return [(x[0][a:a + n], x[1][s:s - (-n // 32)]) for a, s, n in zip(self.at, self.sat, self.sizes)]
        return [x[a:a + n] for a, n in zip(self.at, self.sizes)]

    def tensors(self, hg):
        return hg.adamw_tensors(*(self.parts(k) for k in "pgmv"), masters=self.parts("w"))

    def check(self, t, seed=0, lr=LR, gs=None, place0=0, **kw):
        """The device's buffers against a step of what is on the CPU."""
        for i, (a, s, n) in enumerate(zip(self.at, self.sat, self.sizes)):
            sl, bl = slice(a, a + n), slice(s, s - (-n // 32))
            g = self.g[sl].float().numpy()
            old = lambda x: values(x[0][sl], x[1][bl]) if self.bits == 8 else x[sl].numpy()  # noqa: E731
            w = (self.p[sl].float() if self.w is None else self.w[sl]).numpy()
            m, v, new, err = step_of(g, old(self.m), old(self.v), w, t, lr, gs, **kw)
            got = self.dev["p" if self.w is None else "w"][sl].cpu()
            none = new.isnan()
            assert torch.equal(got.isnan(), none)
            ref.check(got[~none], new[~none], err[~none], f"weight {i}")
            if self.w is not None:
                assert torch.equal(self.dev["p"][sl].cpu()[~none], got.to(self.t)[~none])
                self.w[sl] = got
            self.p[sl] = self.dev["p"][sl].cpu()
            if self.bits == 32:
                self.m[sl], self.v[sl] = torch.from_numpy(m), torch.from_numpy(v)
            else:
                r = bits(seed, t, place0(i) if callable(place0) else i + place0, 0, n)
                for x, y, q, keep in ((self.m, m, r & np.uint32(0xffff), False), (self.v, v, r >> np.uint32(16), True)):
                    c, e = rounded(y, q, keep)
                    x[0][sl], x[1][bl] = torch.from_numpy(c), torch.from_numpy(e)
        # everything, gaps among it
        for k in "pwgmv":
            mine, dev = getattr(self, k), self.dev[k]
            pairs = zip(mine, dev) if isinstance(mine, tuple) else [] if mine is None else [(mine, dev)]
            for j, (x, y) in enumerate(pairs):
                y = y.cpu()
                same = (x == y) | ((x != x) & (y != y))
                if isinstance(mine, tuple) and j == 0:
                    same |= ((x & 127) == 127) & ((y & 127) == 127)               # NaN, of either sign
                assert same.all(), (k, int((~same).sum()), [(int(i), x[i].item(), y[i].item()) for i in (~same).nonzero()[:4, 0]])


SIZES = [1, 0, 31, 32, 33, 7, 8, 9, 2047, 2048, 2049, 100, 8192, 8193, 5000]


@pytest.mark.parametrize("t,bits,master", [(F32, 32, False), (F32, 8, False), (BF16, 32, False), (BF16, 8, True),
                                           (F16, 8, False), (F16, 32, True), (BF16, 32, True), (BF16, 8, False)])
@pytest.mark.parametrize("gap,shift", [(0, 0), (3, 1)])
def test_step(hg, t, bits, master, gap, shift):
    print(f"[adamw] {t} {bits} master={master} gap={gap}", flush=True)
    b = Buffers(SIZES, t, bits, master, gap, shift=shift)
    tensors = b.tensors(hg)
    for step in (1, 2, 1000):
        hg.adamw(tensors, step, LR, (B1, B2), EPS, DECAY, seed=step * 77 + (1 << 40))
        b.check(step, step * 77 + (1 << 40))


@pytest.mark.parametrize("count", [47, 48, 49, 97, 300])
def test_many_tensors(hg, count):
    """More than a launch takes, and places in the call that go on."""
    rng = np.random.default_rng(count)
    b = Buffers([int(n) for n in rng.integers(0, 3000, count)], BF16, 8, True)
    hg.adamw(b.tensors(hg), 5, LR, (B1, B2), EPS, DECAY, seed=3)
    b.check(5, 3)


@pytest.mark.parametrize("bits", [8, 32])
def test_large_tensors(hg, bits):
    """Long pieces."""
    b = Buffers([5000000, 3000001, 77], BF16, bits, False)
    hg.adamw(b.tensors(hg), 7, LR, (B1, B2), EPS, DECAY, seed=9)
    b.check(7, 9)


@pytest.mark.parametrize("gtype", [F16, BF16, F32])
@pytest.mark.parametrize("t", [F16, BF16, F32])
def test_gradients_of_another_type(hg, t, gtype):
    b = Buffers([3000, 65], t, 32, False, gtype=gtype)
    hg.adamw(b.tensors(hg), 4, LR, (B1, B2), EPS, DECAY)
    b.check(4)


@pytest.mark.parametrize("kw", [dict(b1=0.0, b2=0.0, eps=1e-3), dict(b1=0.5, b2=0.9999, decay=0.0), dict(eps=0.0)])
def test_other_rates(hg, kw):
    b = Buffers([3000, 65], F32, 32, False)
    d = dict(b1=B1, b2=B2, eps=EPS, decay=DECAY) | kw
    hg.adamw(b.tensors(hg), 3, LR, (d["b1"], d["b2"]), d["eps"], d["decay"])
    b.check(3, **d)


def test_factors_and_device_step(hg):
    """lr and gradients multiplied on the device; a step of 0 there changes nothing."""
    b = Buffers([3000, 65], BF16, 8, True)
    tensors = b.tensors(hg)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    factors = torch.tensor([0.25, 0.5], device=DEV)
    before = [x.clone() for k in "pw" for x in [b.dev[k]]] + [x.clone() for k in "mv" for x in b.dev[k]]
    hg.adamw(tensors, step, LR, (B1, B2), EPS, DECAY, factors=factors)
    after = [b.dev[k] for k in "pw"] + [x for k in "mv" for x in b.dev[k]]
    assert all(torch.equal(x, y) for x, y in zip(before, after))
    step += 6
    hg.adamw(tensors, step, LR, (B1, B2), EPS, DECAY, factors=factors, seed=1)
    b.check(6, 1, lr=LR * 0.25, gs=0.5)


@pytest.mark.parametrize("t,bits,master", [(BF16, 8, False), (F32, 32, False), (BF16, 8, True)])
def test_infinite_and_extreme_gradients(hg, t, bits, master):
    """A NaN or an infinity stays in its element; zeros, the smallest and the largest gradients."""
    b = Buffers([320, 33], t, bits, master)
    for x in (b.g, b.dev["g"]):
        x[3], x[40], x[41] = float("nan"), float("inf"), -float("inf")
        x[64:96] = 0
        x[96:128] = 1e-20
        x[128:160] = 1e15
        x[160:192] = 1e18
        x[192] = 1e-30
        x[352] = float("nan")
    if bits == 8:
        for x in (b.m, b.v, b.dev["m"], b.dev["v"]):
            x[0][64:160] = 0
            x[1][2:5] = 0
    tensors = b.tensors(hg)
    for step in (1, 2):
        hg.adamw(tensors, step, LR, (B1, B2), EPS, DECAY, seed=8)
        b.check(step, 8)


def test_graph(hg):
    """A captured step, its number counted up on the device, with other gradients in every replay."""
    b = Buffers([3000, 65, 9000], BF16, 8, True)
    tensors = b.tensors(hg)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step += 1
        hg.adamw(tensors, step, LR, (B1, B2), EPS, DECAY, seed=11)
    assert int(step) == 0
    for t in range(1, 5):
        b.g = (0.1 * torch.randn(len(b.g), generator=torch.Generator().manual_seed(t))).to(BF16)
        b.dev["g"].copy_(b.g)
        graph.replay()
        torch.cuda.synchronize()
        b.check(t, 11)


def test_past_32_bits(hg):
    """A tensor of more than 2^32 elements: the end of it."""
    n, tail = (1 << 32) + 1000, 1000
    g = torch.Generator().manual_seed(0)
    p, gr = (torch.zeros(n, dtype=BF16, device=DEV) for _ in range(2))
    m, v = hg.adamw_state(p, 8)
    w0, g0 = torch.randn(tail, generator=g).to(BF16), torch.randn(tail, generator=g).to(BF16)
    p[-tail:], gr[-tail:] = w0.to(DEV), g0.to(DEV)
    hg.adamw(hg.adamw_tensors([p], [gr], [m], [v]), 1, LR, (B1, B2), EPS, DECAY, seed=2)
    zero = np.zeros(tail, np.float32)
    nm, nv, new, err = step_of(g0.float().numpy(), zero, zero, w0.float().numpy(), 1)
    ref.check(p[-tail:], new, err, "param")
    r = bits(2, 1, 0, 1 << 32, tail)
    for (codes, scales), y, q, keep in ((m, nm, r & np.uint32(0xffff), False), (v, nv, r >> np.uint32(16), True)):
        c, e = rounded(y, q, keep)
        assert np.array_equal(codes[-tail:].cpu().numpy(), c) and np.array_equal(scales[-len(e):].cpu().numpy(), e)
        assert not codes[:100].any()


def test_eight_bit_moments_follow(hg):
    """Random rounding leaves no drift: with gradients of one size v goes the way of its fp32 sum on average, where
    rounding to nearest would leave it where a step changes less than half a code's distance.

    A code is 2^-3 of a value at most, and a step moves v by d = 0.001·(1 - v), so up by a code with probability d over
    that distance: a variance of at most d·v/8 a step, which decays with 0.998: at most 0.001·v/8/0.002 = v/16, a
    standard deviation of v/4.  The mean of 65536 elements is off by less than 5·v/4/256."""
    n = 65536
    p = torch.zeros(n, device=DEV)
    g = torch.ones(n, device=DEV)
    m, v = hg.adamw_state(p, 8)
    tensors = hg.adamw_tensors([p], [g], [m], [v])
    for t in range(1, 1501):
        hg.adamw(tensors, t, 0.0, (B1, B2), EPS, 0.0, seed=4)
        if t in (300, 1500):
            got = values(v[0].cpu(), v[1].cpu()).astype(np.float64)
            want = 1 - B2 ** t
            assert abs(got.mean() - want) < 5 * want / 4 / 256, t
            assert got.std() < 0.3 * want


def test_state_is_a_checkpoint(hg):
    """8-bit moments of a matrix are read as hg_checkpoint8_read does."""
    p = torch.randn(40, 96, device=DEV)
    m, v = hg.adamw_state(p, 8)
    hg.adamw(hg.adamw_tensors([p], [torch.randn(40, 96, device=DEV)], [m], [v]), 1)
    for codes, scales in (m, v):
        x = hg.checkpoint8_read(codes, scales.view(40, 3), torch.empty(40, 96, dtype=BF16, device=DEV))
        assert torch.equal(x.cpu().float().flatten(), torch.from_numpy(values(codes.cpu().flatten(), scales.cpu())))


def test_a_training_step(hg):
    """The head's product, log probabilities, their gradient, the layer's gradient and the step, after one another:
    gradients against differences of the loss in 64 bits, the weight against the step of the gradient that there is."""
    M, V, K = 48, 500, 64
    g = torch.Generator().manual_seed(0)
    X, W = torch.randn(M, K, generator=g).to(BF16), (torch.randn(V, K, generator=g) / 8).to(BF16)
    tokens = torch.randint(0, V, (M,), generator=g)
    x, w, tok = X.to(DEV), W.to(DEV), tokens.to(DEV)
    new = lambda *s, t=F32: torch.empty(*s, dtype=t, device=DEV)  # noqa: E731
    logits = hg.linear(x, w, new(M, V, t=BF16))
    logp, entropy, stats = new(M), new(M), new(M, 2)
    hg.logprobs(logits, tok, logp=logp, entropy=entropy, stats=stats)
    hg.logprobs_grad(logits, tok, stats, logits, dlogp=torch.full((M,), -1.0 / M, device=DEV))
    dw = new(V, K)
    hg.linear_grad(logits, w, x, dW=dw)
    master = W.float().to(DEV)
    m, v = hg.adamw_state(master, 8)
    hg.adamw(hg.adamw_tensors([w], [dw], [m], [v], masters=[master]), 1, LR, (B1, B2), EPS, DECAY, seed=5)

    def loss(at):
        return -torch.log_softmax(X.double() @ at.t(), 1).gather(1, tokens[:, None]).mean()

    way = torch.randn(V, K, generator=g, dtype=torch.float64)
    h = 1e-4
    change = (loss(W.double() + h * way) - loss(W.double() - h * way)) / (2 * h)
    got = (dw.cpu().double() * way).sum()
    # logits and their gradient are rounded to bf16: each moves the gradient by at most 2^-8 of its size, logits of size s
    # their p by s·2^-8; the sum of V·K products with `way` of the magnitudes bounds both
    z = X.double() @ W.double().t()
    p = torch.softmax(z, 1)
    one = torch.zeros(M, V).double().scatter_(1, tokens[:, None], 1.0)
    dz = (p * (2 * z.abs().amax(1, keepdim=True)) + (p - one).abs()) / M * 2.0 ** -8
    lim = (dz * (X.double() @ way.t()).abs()).sum() + h ** 2 * 1e4
    assert (got - change).abs() < lim
    zero = np.zeros(V * K, np.float32)
    gr = dw.cpu().flatten().numpy()
    nm, _, want, err = step_of(gr, zero, zero, W.float().flatten().numpy(), 1)
    ref.check(master.flatten(), want, err, "master")
    r = bits(5, 1, 0, 0, V * K)
    assert np.array_equal(m[0].cpu().flatten().numpy(), rounded(nm, r & np.uint32(0xffff), False)[0])


@pytest.mark.parametrize("t,bits,master,most", [(F32, 32, False, 83), (BF16, 32, True, 69), (BF16, 8, False, 59), (F16, 8, True, 51)])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_as_many_as_a_launch_takes(hg, t, bits, master, most, more):
    """Of each kind of tensor, and one less and one more."""
    b = Buffers([1 + 37 * i % 101 for i in range(most + more)], t, bits, master)
    hg.adamw(b.tensors(hg), 4, LR, (B1, B2), EPS, DECAY, seed=6)
    b.check(4, 6)


def test_kinds_in_turn(hg):
    """Tensors of all kinds in one call, in an order in which none follows its like."""
    kinds = [(F32, 32, False), (BF16, 8, True), (F16, 8, False), (BF16, 32, True), (F16, 32, False), (F32, 8, False)]
    bs = [Buffers([1 + (i * 53 + k * 7) % 90 for i in range(20)], *kind, seed=k) for k, kind in enumerate(kinds)]
    lists = {key: [b.parts(key) or [None] * 20 for b in bs] for key in "pgmvw"}
    turn = {key: [x[i] for i in range(20) for x in xs] for key, xs in lists.items()}
    hg.adamw(hg.adamw_tensors(*(turn[k] for k in "pgmv"), masters=turn["w"]), 3, LR, (B1, B2), EPS, DECAY, seed=8)
    for k, b in enumerate(bs):
        b.check(3, 8, place0=lambda i: len(kinds) * i + k)


@pytest.mark.parametrize("size", [1e-15, 1e-18, 3e-19, 1e-19, 1e-20, 3e-21])
def test_second_moments_below_the_least_normal_number(hg, size):
    """With eps = 0 the quotient still is that of the moments, however small they are."""
    n, f = 97, np.float32
    g = (size * np.linspace(0.5, 2.0, n)).astype(f)
    p, m, v = (torch.zeros(n, device=DEV) for _ in range(3))
    hg.adamw(hg.adamw_tensors([p], [torch.from_numpy(g).to(DEV)], [m], [v]), 1, 0.5, (B1, B2), 0.0, 0.0)
    zero = np.zeros(n, f)
    M, V, new, err = step_of(g, zero, zero, zero, 1, 0.5, eps=0.0, decay=0.0)
    assert torch.equal(m.cpu(), torch.from_numpy(M)) and torch.equal(v.cpu(), torch.from_numpy(V))
    # (v times its factor, below the least normal number, is off by half of the least step)
    q = V.astype(np.float64) / (1 - B2)
    err = err + torch.from_numpy(np.where(q > 0, 0.5 * 2.0 ** -149 / np.maximum(q, 2.0 ** -149), 0)) * new.abs()
    some = torch.from_numpy(V > 0)
    ref.check(p.cpu()[some], new[some], err[some], "weight")


@pytest.mark.parametrize("small", [1e-15, 1e-17, 1e-10])
def test_a_tiny_second_moment_beside_a_huge_one(hg, small):
    """In one block of 32, a second moment above 0 never becomes 0, however far below the block's largest it is: the
    quotient 1e-33 / 2^102 itself leaves fp32."""
    n = 64
    g = torch.zeros(n)
    g[0], g[1:20], g[32:50] = 1e18, small, small
    p = torch.zeros(n, device=DEV)
    m, v = hg.adamw_state(p, 8)
    tensors = hg.adamw_tensors([p], [g.to(DEV)], [m], [v])
    for t in range(1, 4):
        hg.adamw(tensors, t, LR, (B1, B2), EPS, DECAY, seed=t)
        codes = v[0].cpu()
        assert codes[0] > 0x70 and (codes[1:20] == 1).all(), codes[:32]        # the least code, 2^-9 of the scale
        assert (codes[32:50] > 1).all() and not codes[20:32].any() and not codes[50:].any()


@pytest.mark.parametrize("t,bits,master", [(F32, 32, False), (F32, 8, False), (BF16, 8, True), (BF16, 32, True)])
def test_gradients_whose_square_leaves_fp32(hg, t, bits, master):
    """What the header says of them, beside elements that go on as ever."""
    b = Buffers([200], t, bits, master)
    at, inf = [5, 40, 41, 199], 70
    for x in (b.g, b.dev["g"]):
        x[at], x[inf] = 2e19, -float("inf")
    tensors = b.tensors(hg)
    for step in (1, 2, 3):
        hg.adamw(tensors, step, LR, (B1, B2), EPS, DECAY, seed=2)
        before = (b.p if b.w is None else b.w)[at].float().numpy()
        b.check(step, 2)
        w = b.dev["p" if b.w is None else "w"].cpu().float()
        v = b.v if bits == 32 else torch.from_numpy(values(b.v[0], b.v[1]))
        assert w[inf].isnan() and w.isfinite().sum() == (199 if bits == 32 or step == 1 else 195)
        if bits == 32:
            assert v[at].isinf().all() and v[inf].isinf()
            # (lr·decay and its product with the weight are rounded, and the result, to the param's type last)
            want = torch.from_numpy(before * (1 - LR * DECAY))
            assert ((w[at] - want).abs() <= 4 * U * want.abs() + (0 if t == F32 or master else ref.half(t) * want.abs())).all()
        else:
            assert v[at].isnan().all() and v[inf].isnan()


@pytest.mark.parametrize("t", [(1 << 32) + 5, (1 << 40) - 1])
def test_steps_past_32_bits(hg, t):
    """Both halves of the step's number go into the random bits; from the host and from the device."""
    b = Buffers([3000, 65], BF16, 8, True)
    tensors = b.tensors(hg)
    hg.adamw(tensors, t, LR, (B1, B2), EPS, DECAY, seed=(1 << 64) - 3)
    b.check(t, (1 << 64) - 3)
    hg.adamw(tensors, torch.tensor([t + 1], device=DEV), LR, (B1, B2), EPS, DECAY, seed=-3)
    b.check(t + 1, (1 << 64) - 3)


def test_two_steps_at_once(hg):
    """Of different tensors on two streams, over and over."""
    bs = [Buffers([5000, 65, 33], BF16, 8, True, seed=i) for i in (0, 1)]
    streams, tensors = [torch.cuda.Stream() for _ in bs], [b.tensors(hg) for b in bs]
    torch.cuda.synchronize()
    for t in range(1, 5):
        for stream, x in zip(streams, tensors):
            with torch.cuda.stream(stream):
                hg.adamw(x, t, LR, (B1, B2), EPS, DECAY, seed=t)
    torch.cuda.synchronize()
    for b in bs:
        dev = {k: b.dev[k] for k in "pwmv"}
        again = Buffers([5000, 65, 33], BF16, 8, True, seed=bs.index(b))
        x = again.tensors(hg)
        for t in range(1, 5):
            hg.adamw(x, t, LR, (B1, B2), EPS, DECAY, seed=t)
            again.check(t, t)
        for k, v in dev.items():
            for p, q in zip(v if isinstance(v, tuple) else (v,), again.dev[k] if isinstance(v, tuple) else (again.dev[k],)):
                assert torch.equal(p, q), k
