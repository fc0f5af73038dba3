"""What stands around the linear layer when a model is served with adapters and trained: what is measured, and the plain forms.

Four kinds of case:

    adapters   Y = act(X·Wᵀ + bias + s_g·(X·A_gᵀ)·B_gᵀ) + R: the low-rank adapters of many requests beside a
               shared projection, row i of X with the adapter g = which[i] (outside 0 .. G-1: with none)
    logprobs   of every row of logits the log probability of a given token, the entropy, the statistics of the
               softmax, and the most probable tokens with theirs
    dlogits    the gradient of the two: dx = scale·(dl·(1[token] - p) - dh·p·(log p + H))
    adamw      a step of AdamW over many tensors, the moments in 32 bits or as 8-bit checkpoints

8-bit moments: e4m3 codes, one power-of-two scale for every 32 consecutive elements, as the 8-bit checkpoints of
bf16 values, but rounded at random: up or down by the distance to either code, the random bits a hash of seed, step,
tensor and element.  A positive second moment is never rounded to zero.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK = 32
#: no case multiplies more than the largest listed one, has more logits or more elements
MOST_PRODUCT = 8192 * 4096 * 4096
MOST_LOGITS = 8192 * 50264
MOST_ELEMENTS = 1 << 27
LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.01


def _adapters(name, M, N, K, rank, adapters, type, order, act="none", bias=False, residual=False, out="16"):
    return {"name": name, "op": "adapters", "M": M, "N": N, "K": K, "rank": rank, "adapters": adapters, "type": type,
            "order": order, "act": act, "bias": bias, "residual": residual, "out": out}


def _logprobs(name, M, V, type, top, entropy=True, mask=False, scale=1.0):
    return {"name": name, "op": "logprobs", "M": M, "V": V, "type": type, "top": top, "entropy": entropy, "mask": mask,
            "scale": scale}


def _dlogits(name, M, V, type, entropy=True, scale=1.0):
    return {"name": name, "op": "dlogits", "M": M, "V": V, "type": type, "entropy": entropy, "scale": scale}


def _adamw(name, tensors, size, type, bits, master=False, packed=False):
    return {"name": name, "op": "adamw", "tensors": tensors, "size": size, "type": type, "bits": bits, "master": master,
            "packed": packed}


def listed():
    return [
        # one request's next token through a projection with its adapter
        _adapters("token", 1, 4096, 4096, 16, 8, "bf16", "single"),
        # the next tokens of 64 requests, each with an adapter of its own
        _adapters("tokens64", 64, 4096, 4096, 16, 64, "f16", "single", residual=True),
        # prompts of many requests after each other, tokens of running requests between them
        _adapters("prompts", 8192, 4096, 4096, 16, 16, "bf16", "runs"),
        # rows that are not 16-byte aligned, rows of different adapters next to each other
        _adapters("odd", 333, 1111, 777, 9, 5, "bf16", "single", act="silu", bias=True),
        # one token's distribution: its log probability, the entropy, twenty alternatives
        _logprobs("next_token", 1, 50264, "bf16", 20),
        # a training batch's log probabilities with five alternatives
        _logprobs("batch", 8192, 50264, "bf16", 5),
        # fp32 logits of odd length, part of the vocabulary masked out, sampled at a temperature
        _logprobs("masked", 333, 32003, "f32", 8, mask=True, scale=1.25),
        # the gradient of batch, with an entropy bonus
        _dlogits("dbatch", 8192, 50264, "bf16"),
        # a small head's, fp32
        _dlogits("dsmall", 64, 1000, "f32", entropy=False),
        # the adapters of a model: many small tensors, fp32 all through
        _adamw("adapters_step", 64, 65536, "f32", 32),
        # a layer's weights in bf16 with fp32 masters, moments in 8 bits
        _adamw("layer_step", 4, 33554432, "bf16", 8, master=True),
        # fp16 weights one after the other in a buffer, at odd places, moments in 8 bits
        _adamw("packed_step", 11, 100003, "f16", 8, packed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A layer's width: two in three are multiples of 64, the others any number."""
    n = _log(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 2 / 3 else n


def draw(rng):
    op = rng.choice(("adapters", "adapters", "logprobs", "dlogits", "adamw"))
    if op == "adapters":
        while True:
            M, N, K = _log(rng, 1, 8192), _width(rng, 64, 16384), _width(rng, 64, 16384)
            if M * N * K <= MOST_PRODUCT:
                break
        rank = rng.choice((8, 16, 32, 64)) if rng.random() < 0.75 else rng.randint(1, 64)
        return {"op": op, "M": M, "N": N, "K": K, "rank": rank, "adapters": _log(rng, 1, 64),
                "type": rng.choice(("f16", "bf16")), "order": rng.choice(("single", "runs", "runs")),
                "act": rng.choice(("none", "none") + ACTS), "bias": rng.random() < 0.4, "residual": rng.random() < 0.3,
                "out": rng.choice(("16", "16", "f32"))}
    if op == "adamw":
        tensors, size = _log(rng, 1, 256), _log(rng, 64, 1 << 26)
        type = rng.choice(("f16", "bf16", "f32"))
        return {"op": op, "tensors": tensors, "size": min(size, MOST_ELEMENTS // tensors), "type": type,
                "bits": rng.choice((8, 32)), "master": type != "f32" and rng.random() < 0.5, "packed": rng.random() < 0.3}
    V = _log(rng, 64, 131072)
    c = {"op": op, "M": min(_log(rng, 1, 8192), MOST_LOGITS // V), "V": V, "type": rng.choice(("f16", "bf16", "f32")),
         "entropy": rng.random() < 0.6, "scale": rng.choice((1.0, 1.0, 0.5, 1.25))}
    if op == "logprobs":
        c.update(top=rng.choice((0, 1, 5, 8, 20, 32)), mask=rng.random() < 0.3)
    return c


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _activation(gen, M, K, t):
    """Activations: normal, a few channels far larger than the rest, as a trained model's are."""
    x = _normal(gen, M, K)
    big = torch.rand(K, generator=gen, device=DEV) < 0.004
    return (x * torch.where(big, 12.0, 1.0)).to(t)


def _which(gen, M, adapters, order):
    """The rows' adapters, -1 for none: each row's own, or runs of prompts and single tokens."""
    ids = torch.randint(-1, adapters, (M,), generator=gen, device=DEV)
    ids[0].clamp_(min=0)
    if order == "single":
        return ids
    # about one row in 128 begins another request's
    first = torch.rand(M, generator=gen, device=DEV) < 1 / 128
    first[0] = True
    return ids[first.nonzero()[:, 0]][first.cumsum(0) - 1].contiguous()


def _sizes(case):
    """Every other tensor is a vector or a smaller matrix."""
    return [case["size"] if i % 2 == 0 else case["size"] // 29 + i for i in range(case["tensors"])]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[case["type"]]
    op = case["op"]
    s = {"case": case}

    def room(key, *shape, type=t):
        s[key] = torch.empty(*shape, dtype=type, device=DEV)

    if op == "adapters":
        M, N, K, r, G = case["M"], case["N"], case["K"], case["rank"], case["adapters"]
        s["X"] = _activation(gen, M, K, t)
        s["W"] = (_normal(gen, N, K) / math.sqrt(K)).to(t)
        s["A"] = (_normal(gen, G, r, K) / math.sqrt(K)).to(t)
        s["B"] = (0.1 * _normal(gen, G, N, r)).to(t)
        s["s"] = 0.5 + 1.5 * torch.rand(G, generator=gen, device=DEV)
        s["which"] = _which(gen, M, G, case["order"])
        out = TYPES["f32"] if case["out"] == "f32" else t
        s["bias"] = 0.1 * _normal(gen, N) if case["bias"] else None
        s["R"] = _normal(gen, M, N).to(out) if case["residual"] else None
        room("Y", M, N, type=out)
        return s
    if op == "adamw":
        sizes = _sizes(case)
        step = 1 if case["packed"] else 64
        at = [0]
        for n in sizes:
            at.append(at[-1] + -(-n // step) * step)
        total = at[-1]
        s["at"], s["sizes"], s["t"], s["seed"] = at, sizes, 100, seed

        def parts(x):
            return [x[a:a + n] for a, n in zip(at, sizes)]

        master = 0.02 * _normal(gen, total)
        s["P"] = master.to(t)
        s["W"] = master if case["master"] else None
        g = 0.01 * _normal(gen, total) * torch.exp(_normal(gen, total))
        s["G"] = g.to(t)
        m, v = 0.2 * g.roll(1), g.roll(2).square() + 1e-6 * torch.rand(total, generator=gen, device=DEV)
        del g
        s["p"], s["g"], s["w"] = parts(s["P"]), parts(s["G"]), parts(s["W"]) if case["master"] else None
        if case["bits"] == 32:
            s["M"], s["V"] = m, v
            s["m"], s["v"] = parts(m), parts(v)
            return s
        blocks = [0]
        for n in sizes:
            blocks.append(blocks[-1] + -(-n // BLOCK))
        for key, x in (("m", m), ("v", v)):
            codes = torch.zeros(total, dtype=torch.uint8, device=DEV)
            scales = torch.zeros(blocks[-1], dtype=torch.uint8, device=DEV)
            s[key.upper()] = codes, scales
            s[key] = [(codes[a:a + n], scales[b:b + -(-n // BLOCK)]) for a, n, b in zip(at, sizes, blocks)]
            half = torch.full((), 1 << 15, dtype=torch.int64, device=DEV)
            for (c, e), y in zip(s[key], parts(x)):
                new = _codes(y, half, key == "v")
                c.copy_(new[0])
                e.copy_(new[1])
        return s
    M, V = case["M"], case["V"]
    x = 2.5 * _normal(gen, M, V)
    s["tokens"] = torch.randint(0, V, (M,), generator=gen, device=DEV)
    # the token that was sampled or is to be learnt is mostly a probable one
    x.scatter_add_(1, s["tokens"][:, None], 6 * torch.rand(M, 1, generator=gen, device=DEV))
    if case.get("mask"):
        # a grammar allows part of the vocabulary (the token among it) in some rows
        out = (torch.rand(V, generator=gen, device=DEV) < 0.3) & (torch.rand(M, 1, generator=gen, device=DEV) < 0.5)
        x.masked_fill_(out.scatter(1, s["tokens"][:, None], False), -math.inf)
    s["X"] = x.to(t)
    # positions that are not to be counted (padding, prompts)
    s["tokens"][torch.rand(M, generator=gen, device=DEV) < 0.05] = -1
    del x
    if op == "logprobs":
        room("logp", M, type=torch.float32)
        room("stats", M, 2, type=torch.float32)
        s["entropy"] = torch.empty(M, device=DEV) if case["entropy"] else None
        k = case["top"]
        s["top"] = (torch.empty(M, k, dtype=torch.int64, device=DEV), torch.empty(M, k, device=DEV)) if k else None
        return s
    _, s["entropy"], s["stats"] = _statistics(s["X"], s["tokens"], case["scale"])
    s["dl"] = _normal(gen, M) / M
    s["dh"] = 0.01 * _normal(gen, M) / M if case["entropy"] else None
    room("dX", M, V)
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


def _plain_adapters(s):
    c = s["case"]
    G, r, K = s["A"].shape
    x = s["X"].float()
    # every row's product with all adapters, then its own alone, is one matrix product each way
    mine = (s["which"][:, None] == torch.arange(G, device=x.device)) * s["s"]
    t = (x @ s["A"].float().view(G * r, K).t()).view(-1, G, r) * mine[:, :, None]
    z = x @ s["W"].float().t() + t.view(-1, G * r) @ s["B"].float().transpose(1, 2).reshape(G * r, -1)
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, c["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(s["Y"].dtype)


def _statistics(logits, tokens, scale):
    """(log p of the tokens, 0 where there is none; entropy; [largest logit, log of the sum of exp of the others' distances])"""
    x = logits.float()
    top = x.amax(1)
    d = (x - top[:, None]) * scale
    p = torch.exp(d)
    total = p.sum(1)
    logsum = torch.log(total)
    entropy = logsum - torch.where(p > 0, d * p, torch.zeros_like(p)).sum(1) / total
    at = tokens.clamp(0, x.shape[1] - 1)[:, None]
    logp = torch.where(tokens == at[:, 0], d.gather(1, at)[:, 0] - logsum, torch.zeros_like(top))
    return logp, entropy, torch.stack((top, logsum), 1)


def _plain_logprobs(s):
    c = s["case"]
    logp, entropy, stats = _statistics(s["X"], s["tokens"], c["scale"])
    out = {"logp": logp, "stats": stats}
    if c["entropy"]:
        out["entropy"] = entropy
    if c["top"]:
        # the order of the logits, of equal ones the first, as one whole number each
        x = s["X"].float() + 0.0
        b = x.view(torch.int32)
        key = (b ^ ((b >> 31) & 0x7fffffff)).long() << 32
        key += torch.arange(x.shape[1] - 1, -1, -1, device=x.device)
        ids = x.shape[1] - 1 - (torch.topk(key, c["top"], dim=1).values & 0xffffffff)
        out["top_ids"] = ids
        out["top_logp"] = (x.gather(1, ids) - stats[:, :1]) * c["scale"] - stats[:, 1:]
    return out


def _plain_dlogits(s):
    c = s["case"]
    x = s["X"].float()
    logp = (x - s["stats"][:, :1]) * c["scale"] - s["stats"][:, 1:]
    p = torch.exp(logp)
    at = s["tokens"].clamp(0, x.shape[1] - 1)[:, None]
    dl = torch.where(s["tokens"] == at[:, 0], s["dl"], torch.zeros_like(s["dl"]))[:, None]
    d = -dl * p
    if s["dh"] is not None:
        d -= s["dh"][:, None] * torch.where(p > 0, p * (logp + s["entropy"][:, None]), torch.zeros_like(p))
    d.scatter_add_(1, at, dl)
    return (c["scale"] * d).to(s["X"].dtype)


def _mix(x):
    """A hash of whole numbers below 2^32."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B9) & 0xffffffff
    x = x ^ (x >> 15)
    x = (x * 0xB504F333) & 0xffffffff
    return x ^ (x >> 16)


def _random(seed, step, tensor, n):
    """32 random bits for every element of a tensor (of fewer than 2^32)."""
    key = 0
    for word in (tensor, step & 0xffffffff, step >> 32, seed & 0xffffffff, seed >> 32, 0):
        key = _mix((key + word + 0x9E3779B9) & 0xffffffff)
    return _mix(torch.arange(n, device=DEV) ^ key)


def _codes(x, random, second):
    """x (fp32) as codes and scale bytes; 16 random bits decide between the two nearest codes."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    frac, e = torch.frexp(b.abs().amax(1))                # amax = frac·2^e, 0.5 <= frac < 1; 448 = 0.875·2^9
    e = (e - 9 + (frac > 0.875).to(e.dtype)).clamp(min=-117)
    e = torch.where(frac == 0, torch.full_like(e, -117), e)
    y = torch.ldexp(b.abs(), -e[:, None]).view(-1)[:n]
    low = y < 2.0 ** -6                                   # codes 2^-9 apart, as from 2^-6 to 2^-5
    z = torch.where(low, y + 2.0 ** -6, y).view(torch.int32)
    z = (z + (random.to(torch.int32) << 4) + 8) & ~0xfffff
    q = z.view(torch.float32)
    q = torch.where(low, q - 2.0 ** -6, q)
    if second:
        q = torch.where((y > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return torch.copysign(q, x).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    n = codes.numel()
    v = codes.view(torch.float8_e4m3fn).float()
    return v * torch.ldexp(torch.ones_like(v), scales.int().repeat_interleave(BLOCK)[:n] - 127)


def _plain_step(c, t, seed, i, p, g, w, m, v):
    g = g.float()
    eight = c["bits"] == 8
    old_m, old_v = (_values(*m), _values(*v)) if eight else (m, v)
    new_m = BETA1 * old_m + (1 - BETA1) * g
    new_v = BETA2 * old_v + (1 - BETA2) * (g * g)
    x = p.float() if w is None else w
    mean, square = new_m / (1 - BETA1 ** t), new_v / (1 - BETA2 ** t)
    x = x - LR * (DECAY * x + mean / (torch.sqrt(square) + EPS))
    if w is not None:
        w.copy_(x)
    p.copy_(x)
    if eight:
        h = _random(seed, t, i, g.numel())
        for (codes, scales), new in ((m, _codes(new_m, h & 0xffff, False)), (v, _codes(new_v, h >> 16, True))):
            codes.copy_(new[0])
            scales.copy_(new[1])
    else:
        m.copy_(new_m)
        v.copy_(new_v)


def _stepped(s):
    """The buffers that a step has changed; 8-bit moments as the codes' values and the scale bytes."""
    out = {"P": s["P"]}
    if s["W"] is not None:
        out["W"] = s["W"]
    if s["case"]["bits"] == 32:
        out["M"], out["V"] = s["M"], s["V"]
    else:
        out["M"] = s["M"][0].view(torch.float8_e4m3fn), s["M"][1]
        out["V"] = s["V"][0].view(torch.float8_e4m3fn), s["V"][1]
    return out


def _plain_adamw(s):
    c = s["case"]
    s["t"] += 1
    none = [None] * c["tensors"]
    for i, part in enumerate(zip(s["p"], s["g"], s["w"] or none, s["m"], s["v"])):
        _plain_step(c, s["t"], s["seed"], i, *part)
    return _stepped(s)


# ---- the framework's operators ----

def _framework(s):
    import half_precision_gemm_amd as hg
    c = s["case"]
    op = c["op"]
    if op == "adapters":
        if "work" not in s:
            s["work"] = hg.linear_adapters_workspace(s["X"], s["W"], s["A"])
        return hg.linear_adapters(s["X"], s["W"], s["Y"], s["which"], s["A"], s["B"], scales=s["s"], bias=s["bias"],
                                  act=getattr(hg, "ACT_" + c["act"].upper()), residual=s["R"], work=s["work"])
    if op == "logprobs":
        if "work" not in s:
            s["work"] = hg.logprobs_workspace(s["X"], c["top"])
        hg.logprobs(s["X"], s["tokens"], logp=s["logp"], entropy=s["entropy"], stats=s["stats"], top=s["top"],
                    scale=c["scale"], work=s["work"])
        out = {"logp": s["logp"], "stats": s["stats"]}
        if c["entropy"]:
            out["entropy"] = s["entropy"]
        if c["top"]:
            out["top_ids"], out["top_logp"] = s["top"]
        return out
    if op == "dlogits":
        return hg.logprobs_grad(s["X"], s["tokens"], s["stats"], s["dX"], dlogp=s["dl"], dentropy=s["dh"],
                                entropy=s["entropy"] if s["dh"] is not None else None, scale=c["scale"])
    if "plan" not in s:
        s["plan"] = hg.adamw_tensors(s["p"], s["g"], s["m"], s["v"], masters=s["w"])
    s["t"] += 1
    hg.adamw(s["plan"], s["t"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, seed=s["seed"])
    return _stepped(s)


def run(state):
    if own:
        return _framework(state)
    plain = {"adapters": _plain_adapters, "logprobs": _plain_logprobs, "dlogits": _plain_dlogits, "adamw": _plain_adamw}
    return plain[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    size = 4 if case["type"] == "f32" else 2
    if op == "adapters":
        M, N, K, r = case["M"], case["N"], case["K"], case["rank"]
        # adapters that are in use: at most one a row
        used = min(case["adapters"], M)
        out = 4 if case["out"] == "f32" else 2
        bytes = 2 * (M * K + N * K) + 2 * used * r * (K + N) + 8 * M + out * M * N * (2 if case["residual"] else 1)
        return {"bytes": bytes + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K + 2 * M * r * (N + K)}
    if op == "adamw":
        n = sum(_sizes(case))
        moments = 16 if case["bits"] == 32 else 4 * (1 + 1 / BLOCK)
        # read and written: the weight (with a master: that, and the weight written); read: the gradient
        weight = 8 + size if case["master"] else 2 * size
        return {"bytes": n * (weight + size + moments), "flops": 12 * n}
    M, V = case["M"], case["V"]
    if op == "dlogits":
        return {"bytes": 2 * size * M * V + 28 * M, "flops": 6 * M * V}
    return {"bytes": size * M * V + M * (20 + (4 if case["entropy"] else 0) + 12 * case["top"]), "flops": 4 * M * V}


# ---- the definition in 64 bits ----

def _exact_act(z, act):
    F = torch.nn.functional
    return {"none": lambda v: v.clone(), "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[act](z)


def _exact_adapters(s, case):
    x = s["X"].double()
    z = torch.mm(x, s["W"].double().t())
    for g in range(case["adapters"]):
        rows = (s["which"] == g).nonzero()[:, 0]
        low = torch.mm(x[rows], s["A"][g].double().t())
        z[rows] += s["s"][g].double() * torch.mm(low, s["B"][g].double().t())
    if s["bias"] is not None:
        z = z + s["bias"].double()
    y = _exact_act(z, case["act"])
    return y if s["R"] is None else y + s["R"].double()


def _exact_logprobs(s, case):
    x = s["X"].double()
    logs = torch.log_softmax(x * case["scale"], 1)
    counted = s["tokens"] >= 0
    out = {"logp": torch.where(counted, logs.gather(1, s["tokens"].clamp(min=0)[:, None])[:, 0], 0.0)}
    top = x.max(1).values
    out["stats"] = torch.stack((top, torch.logsumexp(x * case["scale"], 1) - top * case["scale"]), 1)
    if case["entropy"]:
        out["entropy"] = torch.special.entr(logs.exp()).sum(1)
    del x
    if case["top"]:
        ids = s["X"].float().sort(dim=1, descending=True, stable=True).indices[:, :case["top"]].clone()
        out["top_ids"], out["top_logp"] = ids, logs.gather(1, ids)
    return out


def _exact_dlogits(s, case):
    logs = torch.log_softmax(s["X"].double() * case["scale"], 1)
    p = logs.exp()
    dl = torch.where(s["tokens"] >= 0, s["dl"].double(), 0.0)[:, None]
    d = -dl * p
    if s["dh"] is not None:
        d -= s["dh"].double()[:, None] * p * (logs + torch.special.entr(p).sum(1, keepdim=True))
    d.scatter_add_(1, s["tokens"].clamp(min=0)[:, None], dl)
    return d * case["scale"]


def _exact_adamw(s, case):
    t, wide, eight = s["t"] + 1, torch.float64, case["bits"] == 8
    new = {k: s[k].to(wide) for k in ("P",)}
    if s["W"] is not None:
        new["W"] = s["W"].to(wide)
    if not eight:
        new["M"], new["V"] = s["M"].to(wide), s["V"].to(wide)
    for i, (a, n) in enumerate(zip(s["at"], s["sizes"])):
        g = s["g"][i].to(wide)
        m, v = (_values(*s["m"][i]).to(wide), _values(*s["v"][i]).to(wide)) if eight else (s["m"][i].to(wide), s["v"][i].to(wide))
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g.square()
        x = new["P" if s["W"] is None else "W"][a:a + n]
        x = x * (1 - LR * DECAY) - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
        for key, y in (("P", x), ("W", x), ("M", m), ("V", v)):
            if key in new:
                new[key][a:a + n] = y
    if eight:
        # which of two codes is taken goes by random bits and the fp32 sums
        new["M"] = new["V"] = (None, None)
    return new


def exact(case, seed):
    s = prepare(case, seed)
    return {"adapters": _exact_adapters, "logprobs": _exact_logprobs, "dlogits": _exact_dlogits,
            "adamw": _exact_adamw}[case["op"]](s, case)
