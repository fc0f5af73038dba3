"""The linear layer and its training: what is measured, and the plain forms.

Four kinds of case:

    linear   Y = act(X·Wᵀ + bias) + R, optionally with the pre-activation saved
    grad     the layer's gradients dX, dW and dbias from dY and the saved pre-activation
    check    an activation written as an 8-bit checkpoint and read back
    step     a forward and a backward pass of the layer with X and the
             pre-activation kept as 8-bit checkpoints in between

The 8-bit form: e4m3 codes, one power-of-two scale for every 32 consecutive
columns of a row; the exponent e is the smallest with amax <= 448·2^e (fp16:
-15 <= e <= 8, bf16: e >= -117).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK = 32
#: no case multiplies more than the largest listed ones
MOST = 8192 * 16384 * 4096


def _linear(name, M, N, K, type, act, bias=True, residual=False, out="16", save=False):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "type": type, "act": act,
            "bias": bias, "residual": residual, "out": out, "save": save}


def _grad(name, M, N, K, type, act):
    return {"name": name, "op": "grad", "M": M, "N": N, "K": K, "type": type, "act": act}


def _check(name, M, N, type):
    return {"name": name, "op": "check", "M": M, "N": N, "type": type}


def _step(name, M, N, K, type, act):
    return {"name": name, "op": "step", "M": M, "N": N, "K": K, "type": type, "act": act}


def listed():
    return [
        # one token through a projection while text is generated
        _linear("token", 1, 4096, 4096, "bf16", "silu"),
        # sixteen sequences' tokens through the second projection of a feed-forward block, added to the residual stream
        _linear("tokens16", 16, 4096, 16384, "f16", "none", residual=True),
        # a training batch through the first projection, the pre-activation kept for the backward pass
        _linear("batch_up", 8192, 16384, 4096, "bf16", "gelu_tanh", save=True),
        # the repository's ragged size, fp32 output
        _linear("ragged", 1000, 1000, 1000, "f16", "gelu", residual=True, out="f32"),
        # rows that are not 16-byte aligned
        _linear("odd", 333, 1111, 777, "bf16", "relu"),
        # the backward pass of batch_up
        _grad("grad_up", 8192, 16384, 4096, "bf16", "gelu_tanh"),
        # a small layer and a small batch: latency
        _grad("grad_small", 64, 512, 512, "f16", "relu"),
        # a batch whose length is odd
        _grad("grad_odd", 777, 1000, 1304, "f16", "silu"),
        # one short prompt's activations
        _check("check_small", 256, 4096, "f16"),
        # a training batch's activations
        _check("check_large", 8192, 16384, "bf16"),
        # a training step of a layer whose activations are kept in 8 bits
        _step("step", 4096, 8192, 2048, "bf16", "gelu"),
        # the same for a small layer
        _step("step_small", 512, 1024, 1000, "f16", "silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer's width: two in three are multiples of 64, the others any number."""
    n = _log(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 2 / 3 else n


def draw(rng):
    op = rng.choice(("linear", "linear", "grad", "check", "step"))
    type = rng.choice(("f16", "bf16"))
    if op == "check":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _width(rng, 32, 16384), "type": type}
    while True:
        M, N, K = _log(rng, 1, 8192), _width(rng, 64, 16384), _width(rng, 64, 16384)
        if M * N * K <= (MOST if op == "linear" else MOST // 2):
            break
    c = {"op": op, "M": M, "N": N, "K": K, "type": type, "act": rng.choice(ACTS)}
    if op == "linear":
        c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.4, out=rng.choice(("16", "16", "f32")),
                 save=rng.random() < 0.4)
    return c


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _activation(gen, M, K, t):
    """Activations: normal, a few channels far larger than the rest, as a trained model's are."""
    x = _normal(gen, M, K)
    big = torch.rand(K, generator=gen, device=DEV) < 0.004
    return (x * torch.where(big, 12.0, 1.0)).to(t)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[case["type"]]
    op, M, N = case["op"], case["M"], case["N"]
    s = {"case": case}

    def room(key, rows, cols, type=t):
        s[key] = torch.empty(rows, cols, dtype=type, device=DEV)

    def codes(key, rows, cols):
        s[key] = (torch.empty(rows, cols, dtype=torch.uint8, device=DEV),
                  torch.empty(rows, -(-cols // BLOCK), dtype=torch.uint8, device=DEV))

    if op == "check":
        s["X"] = _activation(gen, M, N, t)
        codes("X8", M, N)
        room("back", M, N)
        return s
    K = case["K"]
    s["X"] = _activation(gen, M, K, t)
    s["W"] = (_normal(gen, N, K) / math.sqrt(K)).to(t)
    if op == "linear":
        out = TYPES["f32"] if case["out"] == "f32" else t
        s["bias"] = 0.1 * _normal(gen, N) if case["bias"] else None
        s["R"] = _normal(gen, M, N).to(out) if case["residual"] else None
        room("Y", M, N, out)
        s["Z"] = torch.empty(M, N, dtype=t, device=DEV) if case["save"] else None
        return s
    s["dY"] = (0.05 * _normal(gen, M, N)).to(t)
    room("dX", M, K)
    room("dW", N, K)
    if op == "grad":
        s["Z"] = _normal(gen, M, N).to(t)
        s["dbias"] = torch.empty(N, dtype=torch.float32, device=DEV)
    else:
        room("Y", M, N)
        codes("X8", M, K)
        codes("Z8", M, N)
    return s


# ---- plain forms ----

def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _rounded8(x, half):
    """The values that an 8-bit checkpoint of x (fp32) stands for."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    top = x.abs().amax(2, keepdim=True)
    frac, e = torch.frexp(top)                       # top = frac·2^e, 0.5 <= frac < 1; 448 = 0.875·2^9
    e = e - 9 + (frac > 0.875).to(e.dtype)
    e = torch.where(top == 0, torch.full_like(e, -1000), e)
    e = e.clamp(-15, 8) if half else e.clamp(min=-117)
    v = torch.ldexp(x, -e)
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v)[1].clamp(min=-5) - 4)   # 4 significant bits, 2^-9 at least
    v = torch.round(v / step) * step                 # to even
    if half:
        v = torch.where(e == 8, v.clamp(-240, 240), v)
    return torch.ldexp(v.clamp(-448, 448), e).view(rows, -1)[:, :cols]


def _plain(s):
    c = s["case"]
    t, op = TYPES[c["type"]], c["op"]
    half = t == torch.float16
    x = s["X"].float()
    if op == "check":
        return _rounded8(x, half).to(t)
    w = s["W"].float()
    if op == "linear":
        z = x @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, c["act"])
        if s["R"] is not None:
            y = y + s["R"].float()
        y = y.to(s["Y"].dtype)
        return (y, z.to(t)) if c["save"] else y
    dy = s["dY"].float()
    if op == "grad":
        dz = dy * _slope(s["Z"].float(), c["act"])
        return (dz @ w).to(t), (dz.t() @ x).to(t), dz.sum(0)
    z = x @ w.t()
    y = _act(z, c["act"]).to(t)
    dz = dy * _slope(_rounded8(z, half), c["act"])
    return y, (dz @ w).to(t), (dz.t() @ _rounded8(x, half)).to(t)


# ---- the framework's operators ----

def _framework(s):
    import half_precision_gemm_amd as hg
    c = s["case"]
    op = c["op"]
    if op == "check":
        hg.checkpoint8_write(s["X"], *s["X8"])
        return hg.checkpoint8_read(*s["X8"], s["back"])
    act = getattr(hg, "ACT_" + c["act"].upper())
    if op == "linear":
        if "work" not in s:
            s["work"] = hg.linear_workspace(s["X"], s["W"])
        hg.linear(s["X"], s["W"], s["Y"], bias=s["bias"], act=act, residual=s["R"], Z=s["Z"], work=s["work"])
        return (s["Y"], s["Z"]) if c["save"] else s["Y"]
    if op == "grad":
        if "work" not in s:
            s["work"] = hg.linear_grad_workspace(s["dY"], s["W"], s["X"])
        hg.linear_grad(s["dY"], s["W"], s["X"], Z=s["Z"], act=act, dX=s["dX"], dW=s["dW"], dbias=s["dbias"],
                       work=s["work"])
        return s["dX"], s["dW"], s["dbias"]
    if "work" not in s:
        s["work"] = hg.linear_workspace(s["X"], s["W"])
        s["gwork"] = hg.linear_grad_workspace(s["dY"], s["W"], s["X8"])
    hg.checkpoint8_write(s["X"], *s["X8"])
    hg.linear(s["X"], s["W"], s["Y"], act=act, Z=s["Z8"], work=s["work"])
    hg.linear_grad(s["dY"], s["W"], s["X8"], Z=s["Z8"], act=act, dX=s["dX"], dW=s["dW"], work=s["gwork"])
    return s["Y"], s["dX"], s["dW"]


def run(state):
    return _framework(state) if own else _plain(state)


def work(case):
    op, M, N = case["op"], case["M"], case["N"]
    packed = lambda rows, cols: rows * (cols + -(-cols // BLOCK))  # noqa: E731
    if op == "check":
        return {"bytes": 4 * M * N + 2 * packed(M, N), "flops": 0}
    K = case["K"]
    bytes = 2 * (M * K + N * K)
    if op == "linear":
        out = 4 if case["out"] == "f32" else 2
        bytes += out * M * N * (2 if case["residual"] else 1) + (2 * M * N if case["save"] else 0)
        return {"bytes": bytes + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "grad":
        return {"bytes": 2 * bytes + 4 * M * N + 4 * N, "flops": 4 * M * N * K}
    # X and W read, Y, dX and dW written, dY and W read, both checkpoints written and read
    bytes += 2 * M * N + 2 * (M * K + N * K) + 2 * M * N + 2 * N * K + 2 * packed(M, K) + 2 * packed(M, N)
    return {"bytes": bytes, "flops": 6 * M * N * K}


# ---- the definition in 64 bits ----

def _exact_act(z, act):
    F = torch.nn.functional
    return {"none": lambda v: v.clone(), "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[act](z)


def _exact_dz(z, dy, act):
    z = z.detach().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(_exact_act(z, act), z, dy)[0]


def _exact8(x, type):
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    e = torch.ceil(torch.log2(x.abs().amax(2, keepdim=True) / 448))      # -inf where the block is zero
    e = torch.clamp(e, -15, 8) if type == "f16" else torch.clamp(e, min=-117)
    v = (x * torch.exp2(-e)).clamp(-448, 448).float()
    if type == "f16":
        v = torch.where(e == 8, v.clamp(-240, 240), v)
    return (v.to(torch.float8_e4m3fn).double() * torch.exp2(e)).view(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    x = s["X"].double()
    if op == "check":
        return _exact8(x, case["type"])
    w = s["W"].double()
    if op == "grad":
        dz = _exact_dz(s["Z"].double(), s["dY"].double(), case["act"])
        return torch.mm(dz, w), torch.mm(dz.t(), x), dz.sum(dim=0)
    z = torch.mm(x, w.t())
    if op == "linear":
        if s["bias"] is not None:
            z = z + s["bias"].double()
        y = _exact_act(z, case["act"])
        if s["R"] is not None:
            y = y + s["R"].double()
        return (y, z) if case["save"] else y
    dz = _exact_dz(_exact8(z, case["type"]), s["dY"].double(), case["act"])
    return _exact_act(z, case["act"]), torch.mm(dz, w), torch.mm(dz.t(), _exact8(x, case["type"]))
