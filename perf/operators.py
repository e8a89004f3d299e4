"""What is measured of the training-step operators: layer norm and its
gradient, the gradient norm over a list of tensors, and the AdamW step over a
list of tensors with states in 32 or in 8 bits.

`listed()` names fixed cases, `draw(rng)` makes more of the same ranges,
`prepare(case, seed)` makes what a training program has in hand, `run(state)`
is one call of an operator, `work(case)` what it has to move and compute, and
`exact(case, seed)` the same outputs from the definitions in 64 bits.

The plain forms are elementary torch operations in binary32.  With `own` set,
`run` calls the package's entry points instead.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}

HIDDEN, KV, FFN, WORLD = 3584, 512, 18944, 8  # the transformer layer of the gathers' workload

LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.95, 1e-8, 0.1
BLOCK = 256            # elements of an 8-bit state that share a scale
U32 = 0xFFFFFFFF


# ---------------------------------------------------------------- cases
def layer_sizes(world=1):
    """Elements of each weight of one transformer layer, or of one rank's shard of it."""
    full = [HIDDEN * HIDDEN, KV * HIDDEN, KV * HIDDEN, HIDDEN * HIDDEN,
            FFN * HIDDEN, FFN * HIDDEN, HIDDEN * FFN]
    return [n // world for n in full] + [HIDDEN // world] * 2


def listed():
    return [
        # serving: the norm of one token of each of 8 sequences, where latency is all there is
        dict(name="norm_decode", op="norm", rows=8, cols=HIDDEN, dtype="bf16", wdtype="bf16", pad=0, stats=False),
        # training: forward over a batch of 8 sequences of 4096 tokens, statistics kept for the backward
        dict(name="norm_batch", op="norm", rows=32768, cols=HIDDEN, dtype="bf16", wdtype="fp32", pad=0, stats=True),
        # a head's width that is no multiple of a vector, rows cut out of a wider buffer
        dict(name="norm_odd", op="norm", rows=20011, cols=1027, dtype="fp16", wdtype="fp16", pad=5, stats=True),
        # the gradient of a short sequence, where launches and the reduction of the weight's gradient weigh most
        dict(name="norm_grad_short", op="norm_grad", rows=257, cols=1024, dtype="fp32", wdtype="fp32", pad=0),
        # the gradient of the training batch
        dict(name="norm_grad_batch", op="norm_grad", rows=32768, cols=HIDDEN, dtype="bf16", wdtype="bf16", pad=0),
        # clipping of two small tensors (biases, norm weights)
        dict(name="gradnorm_small", op="gradnorm", dtype="bf16", total=0, count=2, split=0, odd=False),
        # clipping over the gradients of a whole layer
        dict(name="gradnorm_layer", op="gradnorm", dtype="bf16", total=-1, count=9, split=0, odd=False),
        # the step of two small tensors in binary32
        dict(name="adamw_small", op="adamw", dtype="fp32", gdtype="fp32", master=False, total=0, count=2, split=0, odd=False),
        # one rank's shard of a layer: bf16 weights with binary32 masters, clipped
        dict(name="adamw_shard", op="adamw", dtype="bf16", gdtype="bf16", master=True, total=-2, count=9, split=0, odd=False),
        # ragged shards packed one after the other, so that tensors start at any element
        dict(name="adamw_ragged", op="adamw", dtype="fp32", gdtype="fp32", master=False, total=7_000_003, count=61, split=11, odd=True),
        # many small tensors with 8-bit states
        dict(name="adamw8_many", op="adamw8", dtype="bf16", gdtype="fp32", master=True, total=2_500_001, count=150, split=5, odd=True),
        # a whole layer on one rank with 8-bit states and no masters
        dict(name="adamw8_layer", op="adamw8", dtype="bf16", gdtype="bf16", master=False, total=-1, count=9, split=0, odd=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gradnorm", "adamw", "adamw8"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, FFN)
        if rng.random() < 0.6:
            cols = max(64, cols // 8 * 8)
        rows = _log(rng, 1, 65536)
        rows = max(1, min(rows, 100_000_000 // cols))
        c = dict(op=op, rows=rows, cols=cols, dtype=dtype, wdtype=rng.choice([dtype, "fp32"]),
                 pad=rng.choice([0, 0, 8, 3]))
        if op == "norm":
            c["stats"] = rng.random() < 0.5
        return c
    count = _log(rng, 1, 200)
    total = max(count, _log(rng, 2000, 60_000_000))
    c = dict(op=op, dtype=dtype, total=total, count=count, split=rng.randrange(1, 1 << 20), odd=rng.random() < 0.5)
    if op != "gradnorm":
        c["gdtype"] = rng.choice([dtype, "fp32"])
        c["master"] = dtype != "fp32" and rng.random() < 0.5
    return c


def sizes_of(case):
    """Elements of each tensor of the list."""
    if case["total"] == 0:
        return [HIDDEN] * case["count"]
    if case["total"] == -1:
        return layer_sizes()
    if case["total"] == -2:
        return layer_sizes(WORLD)
    r = random.Random(case["split"])
    w = [math.exp(r.uniform(0.0, 5.0)) for _ in range(case["count"])]
    unit = 1 if case["odd"] else 8
    return [max(1, int(case["total"] * x / sum(w)) // unit * unit) for x in w]


def starts_of(case, sizes):
    """Where each tensor starts in its flat buffer, and the buffer's length.
    8-bit states keep whole blocks apart; packed binary32 lists leave no gap."""
    unit = BLOCK if case["op"] == "adamw8" else 1 if case["odd"] else 8
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += -(-n // unit) * unit
    return starts, at


# ---------------------------------------------------------------- what a program has in hand
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(n, scale):
        return torch.randn(n, generator=g, device="cuda") * scale

    s = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        rows, cols, wide = case["rows"], case["cols"], case["cols"] + case["pad"]
        dt, wdt = DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        # activations: a mean and a spread of their own for each row, a few wide columns
        x = normal((rows, wide), 1.0)
        x *= torch.rand((rows, 1), generator=g, device="cuda") * 2 + 0.25
        x += normal((rows, 1), 0.5)
        x[:, :: max(1, cols // 4)] *= 8
        s["x"] = x.to(dt)[:, :cols]
        s["weight"] = (1 + normal(cols, 0.1)).to(wdt)
        s["bias"] = normal(cols, 0.1).to(wdt)
        s["eps"] = 1e-5
        if case["op"] == "norm":
            s["y"] = torch.empty((rows, cols), device="cuda", dtype=dt)
            s["mean"] = torch.empty(rows, device="cuda") if case["stats"] else None
            s["rstd"] = torch.empty(rows, device="cuda") if case["stats"] else None
        else:
            s["dy"] = normal((rows, cols), 0.01).to(dt)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(1) + s["eps"])
            s["dx"] = torch.empty((rows, cols), device="cuda", dtype=dt)
            s["dweight"] = torch.empty(cols, device="cuda", dtype=wdt)
            s["dbias"] = torch.empty(cols, device="cuda", dtype=wdt)
        return s

    sizes = sizes_of(case)
    starts, n = starts_of(case, sizes)
    s["sizes"], s["starts"], s["n"] = sizes, starts, n
    inside = torch.zeros(n + 1, device="cuda", dtype=torch.int32)
    at = torch.tensor(starts, device="cuda")
    end = at + torch.tensor(sizes, device="cuda")
    inside.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    inside.index_add_(0, end, torch.full_like(end, -1, dtype=torch.int32))
    inside = inside.cumsum_(0)[:n].bool()  # false in the gaps between tensors

    def views(flat):
        return [flat[a:a + k] for a, k in zip(starts, sizes)]

    # gradients: magnitudes spread over some decades from one stretch to the next
    spread = torch.exp(torch.randn(n // 1024 + 1, generator=g, device="cuda")).repeat_interleave(1024)[:n]
    grad = normal(n, 1e-3) * spread * inside
    s["grad"] = grad.to(DTYPES[case.get("gdtype", case["dtype"])])
    s["grads"] = views(s["grad"])
    s["max_norm"], s["inv_scale"] = 1.0, 1.0 / WORLD
    s["norm"] = torch.empty(1, device="cuda")
    s["scale"] = torch.full((1,), 0.25 + (seed % 8) / 16, device="cuda")
    if case["op"] == "gradnorm":
        return s
    master = normal(n, 0.02) * inside
    s["param"] = master.to(DTYPES[case["dtype"]])
    s["params"] = views(s["param"])
    s["master"] = master if case["master"] else None
    s["masters"] = views(master) if case["master"] else None
    s["step"] = 10 + seed % 1000
    m = (grad * 0.3 + normal(n, 3e-4) * spread) * inside
    v = (normal(n, 1e-3) * spread).square() * inside
    if case["op"] == "adamw":
        s["m"], s["v"] = m, v
        s["ms"], s["vs"] = views(m), views(v)
        return s
    s["m"], s["m_scale"] = encode(m, None)
    s["r"], s["r_scale"] = encode(v.sqrt(), None, floor=True)
    s["ms"], s["rs"] = views(s["m"]), views(s["r"])
    s["m_scales"] = [s["m_scale"][a // BLOCK:(a + k + BLOCK - 1) // BLOCK] for a, k in zip(starts, sizes)]
    s["r_scales"] = [s["r_scale"][a // BLOCK:(a + k + BLOCK - 1) // BLOCK] for a, k in zip(starts, sizes)]
    return s


# ---------------------------------------------------------------- plain forms
def encode(x, dither, floor=False):
    """Blocks of 256 values as 8-bit floats (4 exponent and 3 mantissa bits) of
    a power-of-two scale that brings the block's largest magnitude into
    [128, 256).  `dither` (16-bit integers) rounds up or down at random in
    proportion; None rounds to the nearest.  `floor`: a positive value is
    never stored as less than the smallest code."""
    x = x.view(-1, BLOCK)
    _, e = torch.frexp(x.abs().amax(1, keepdim=True))
    e = torch.clamp(e - 8, -126, 120)
    scale = torch.ldexp(torch.ones((), device=x.device), e)
    t = torch.ldexp(torch.ones((), device=x.device), -e) * x
    a = t.abs()
    if floor:
        a = torch.where(a > 0, torch.clamp(a, min=2.0 ** -9), a)
    if dither is not None:
        lift = (a < 2.0 ** -6) * 2.0 ** -6
        bits = (a + lift).view(torch.int32) + dither.view(-1, BLOCK) * 16 + 8
        a = (bits & ~0xFFFFF).view(torch.float32) - lift
    return torch.copysign(a, t).to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def decode(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def mix(x):
    """32-bit integer mix of xor-shifts and odd multipliers, in 64-bit integers."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & U32
    x = x ^ (x >> 15)
    x = (x * 0x68E31DA5) & U32
    return x ^ (x >> 16)


def dithers(s, seed):
    """Two 16-bit integers for each element, one for each state, mixed from the
    element's place in its tensor and a key of the tensor and the seed (32-bit
    arithmetic that wraps around; every tensor starts on a whole block)."""
    starts = torch.tensor(s["starts"] + [s["n"]], device="cuda")
    blocks = torch.diff(starts) // BLOCK
    key = mix((seed + torch.arange(1, len(s["starts"]) + 1, device="cuda") * 0x9E3779B9) & U32)
    key = key - starts[:-1] * 0x9E3779B1                       # folds "minus the tensor's start" into the key
    key = torch.repeat_interleave(key, blocks, output_size=s["n"] // BLOCK).to(torch.int32)[:, None]
    h = torch.arange(s["n"], device="cuda", dtype=torch.int32).view(-1, BLOCK) * (0x9E3779B1 - (1 << 32)) + key
    h = h ^ ((h >> 16) & 0xFFFF)
    h = h * 0x7FEB352D
    h = h ^ ((h >> 15) & 0x1FFFF)
    return (h & 0xFFFF).view(-1), ((h >> 16) & 0xFFFF).view(-1)


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + s["eps"])
    y = (c * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(s["x"].dtype)
    return (y, mean, rstd) if s["mean"] is not None else (y,)


def _plain_norm_grad(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dw, db = (dy * xhat).sum(0), dy.sum(0)
    wdy = dy * s["weight"].float()
    c1 = wdy.mean(1, keepdim=True)
    c2 = (wdy * xhat).mean(1, keepdim=True)
    dx = (wdy - c1 - xhat * c2) * s["rstd"][:, None]
    return dx.to(s["x"].dtype), dw.to(s["weight"].dtype), db.to(s["weight"].dtype)


def _plain_gradnorm(s):
    g = s["grad"].float()
    norm = torch.sqrt((g * g).sum()) * s["inv_scale"]
    scale = s["inv_scale"] * torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    scale = torch.where(torch.isfinite(norm), scale, torch.nan)
    return norm.view(1), scale.view(1)


def _plain_adamw(s):
    case, t = s["case"], s["step"]
    s["step"] += 1
    w = s["master"] if case["master"] else s["param"]
    skip = torch.isnan(s["scale"])
    g = s["grad"].float() * s["scale"]
    if case["op"] == "adamw":
        m, v = s["m"], s["v"]
    else:
        m, v = decode(s["m"], s["m_scale"]), decode(s["r"], s["r_scale"])
        v = v * v
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * (1 - BETA2) * g
    r = torch.sqrt(v)
    p = w.float() * (1 - LR * DECAY)
    p = p - m / (r * (1 / math.sqrt(1 - BETA2 ** t)) + EPS) * (LR / (1 - BETA1 ** t))
    if case["master"]:
        torch.where(skip, w, p, out=w)
    s["param"].copy_(torch.where(skip, s["param"], p.to(s["param"].dtype)))
    if case["op"] == "adamw":
        torch.where(skip, s["m"], m, out=s["m"])
        torch.where(skip, s["v"], v, out=s["v"])
        out = [s["param"], s["m"], s["v"]]
    else:
        low, high = dithers(s, t)
        for name, x, d, floor in (("m", m, low, False), ("r", r, high, True)):
            code, scale = encode(x, d, floor)
            s[name].view(torch.uint8).copy_(torch.where(skip, s[name].view(torch.uint8), code.view(torch.uint8)))
            torch.where(skip, s[name + "_scale"], scale, out=s[name + "_scale"])
        out = [s["param"], s["m"], s["m_scale"], s["r"], s["r_scale"]]
    return out + ([s["master"]] if case["master"] else [])


# ---------------------------------------------------------------- the package's operators
def _own_norm(s):
    import allgather_rr_allreduce_gb300 as rr
    c, x, y = s["case"], s["x"], s["y"]
    rr.rr_layer_norm(x, s["weight"], s["bias"], y, s["mean"], s["rstd"], c["rows"], c["cols"], x.stride(0),
                     y.stride(0), s["eps"], c["dtype"], c["wdtype"])
    return (y, s["mean"], s["rstd"]) if s["mean"] is not None else (y,)


def _own_norm_grad(s):
    import allgather_rr_allreduce_gb300 as rr
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(rr.rr_layer_norm_backward_workspace(c["rows"], c["cols"]), device="cuda",
                                     dtype=torch.uint8)
    rr.rr_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                              c["rows"], c["cols"], s["dy"].stride(0), s["x"].stride(0), s["dx"].stride(0),
                              c["dtype"], c["wdtype"], s["workspace"], s["workspace"].numel())
    return s["dx"], s["dweight"], s["dbias"]


def _own_gradnorm(s):
    import allgather_rr_allreduce_gb300 as rr
    if "workspace" not in s:
        s["workspace"] = torch.empty(rr.rr_grad_norm_workspace(len(s["sizes"])), device="cuda", dtype=torch.uint8)
    rr.rr_grad_norm(s["grads"], s["sizes"], s["case"]["dtype"], s["inv_scale"], s["max_norm"], s["norm"], s["scale"],
                    s["workspace"], s["workspace"].numel())
    return s["norm"], s["scale"]


def _own_adamw(s):
    import allgather_rr_allreduce_gb300 as rr
    c, t = s["case"], s["step"]
    s["step"] += 1
    hyper = rr.rr_adamw_hyper(LR, BETA1, BETA2, EPS, DECAY, t)
    if c["op"] == "adamw":
        rr.rr_adamw(s["params"], s["grads"], s["ms"], s["vs"], s["masters"], s["sizes"], c["dtype"], c["gdtype"],
                    hyper, s["scale"])
        out = [s["param"], s["m"], s["v"]]
    else:
        rr.rr_adamw8(s["params"], s["grads"], s["ms"], s["m_scales"], s["rs"], s["r_scales"], s["masters"],
                     s["sizes"], c["dtype"], c["gdtype"], hyper, t, s["scale"])
        out = [s["param"], s["m"], s["m_scale"], s["r"], s["r_scale"]]
    return out + ([s["master"]] if c["master"] else [])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "norm_grad": _own_norm_grad, "gradnorm": _own_gradnorm,
                "adamw": _own_adamw, "adamw8": _own_adamw}[op](state)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "gradnorm": _plain_gradnorm,
            "adamw": _plain_adamw, "adamw8": _plain_adamw}[op](state)


# ---------------------------------------------------------------- work and exact values
def work(case):
    if case["op"] in ("norm", "norm_grad"):
        n, cols = case["rows"] * case["cols"], case["cols"]
        b, wb = BYTES[case["dtype"]], BYTES[case["wdtype"]]
        if case["op"] == "norm":
            return {"bytes": 2 * n * b + 2 * cols * wb + (8 * case["rows"] if case["stats"] else 0), "flops": 8 * n}
        return {"bytes": 3 * n * b + 3 * cols * wb + 8 * case["rows"], "flops": 16 * n}
    sizes = sizes_of(case)
    n = sum(sizes)
    if case["op"] == "gradnorm":
        return {"bytes": n * BYTES[case["dtype"]] + 8, "flops": 2 * n}
    each = BYTES[case["gdtype"]] + (8 + BYTES[case["dtype"]] if case["master"] else 2 * BYTES[case["dtype"]])
    if case["op"] == "adamw":
        return {"bytes": n * (each + 16), "flops": 16 * n}
    return {"bytes": n * (each + 4) + 16 * sum(-(-k // BLOCK) for k in sizes), "flops": 40 * n}


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if case["op"] in ("norm", "norm_grad"):
        x = d["x"]
        if case["op"] == "norm":
            var, mean = torch.var_mean(x, dim=1, unbiased=False)
            rstd = (var + s["eps"]).pow(-0.5)
            y = torch.addcmul(d["bias"], (x - mean[:, None]).mul_(rstd[:, None]), d["weight"])
            return (y, mean, rstd) if case["stats"] else (y,)
        # the chain rule through y = xhat * w + b, xhat = (x - mean) * rstd with mean and rstd functions of x
        xhat = x.sub_(d["mean"][:, None]).mul_(d["rstd"][:, None])
        dweight = torch.einsum("rc,rc->c", d["dy"], xhat)
        dbias = torch.einsum("rc->c", d["dy"])
        dxhat = d["dy"] * d["weight"]
        dot = torch.einsum("rc,rc->r", dxhat, xhat)
        dx = case["cols"] * dxhat - dxhat.sum(1, keepdim=True) - xhat * dot[:, None]
        return dx.mul_(d["rstd"][:, None] / case["cols"]), dweight, dbias
    if case["op"] == "gradnorm":
        norm = torch.linalg.vector_norm(d["grad"]) * s["inv_scale"]
        return norm.view(1), (s["inv_scale"] * min(1.0, s["max_norm"] / (float(norm) + 1e-6)) + 0 * norm).view(1)
    t = s["step"]
    g = d["grad"] * d["scale"]
    eight = case["op"] == "adamw8"
    if eight:
        m = d["m"].view(-1, BLOCK).mul(d["m_scale"][:, None]).view(-1)
        v = d["r"].view(-1, BLOCK).mul(d["r_scale"][:, None]).view(-1).square_()
    else:
        m, v = d["m"], d["v"]
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g.square(), v, BETA2)
    w = d["master"] if case["master"] else d["param"]
    step = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt_() + EPS)
    p = w - LR * DECAY * w - LR * step
    tail = [p] if case["master"] else []
    if not eight:
        return [p, m, v] + tail
    out = [p]
    low, high = dithers(s, t)
    for x, u, floor in ((m, low, False), (v.sqrt(), high, True)):
        x, u = x.view(-1, BLOCK), (u.view(-1, BLOCK).double() + 0.5) / 65536
        top = x.abs().amax(1, keepdim=True)
        e = torch.where(top > 0, torch.log2(torch.where(top > 0, top, 1.0)).floor() - 7, -126.0).clamp_(-126, 120)
        a = x.abs() / torch.exp2(e)
        if floor:
            a = torch.where((a > 0) & (a < 2.0 ** -9), 2.0 ** -9, a)
        q = torch.exp2(torch.log2(torch.clamp(a, min=2.0 ** -6)).floor() - 3)
        out += [(torch.floor(a / q + u) * q * torch.sign(x)).view(-1), torch.exp2(e).view(-1)]
    return out + tail
