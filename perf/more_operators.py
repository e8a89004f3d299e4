"""What is measured of the operators between a model's logits and its new
weights: log-probabilities of tokens and their gradient, the clipped policy
loss, the preference loss over pairs of sequences, the orthogonalisation of
matrices by Newton-Schulz products and the Muon step made of it.

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

HIDDEN, KV, FFN = 3584, 512, 18944  # the transformer layer of the gathers' workload

IGNORED = -100                       # target of a row that takes no part
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.05
BETA, SMOOTHING = 0.1, 0.05
COEFS, STEPS, NORM_EPS = (3.4445, -4.7750, 2.0315), 5, 1e-7
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01


# ---------------------------------------------------------------- cases
def listed():
    return [
        # serving: the log-probabilities of one sampled token of each of 8 sequences, where latency is all there is
        dict(name="logp_tokens", op="logp", rows=8, vocab=131072, dtype="bf16", pad=0, inv_t=1.0),
        # the reference model's log-probabilities of a batch of rollouts; the vocabulary is no multiple of a vector
        dict(name="logp_batch", op="logp", rows=12288, vocab=50021, dtype="fp16", pad=3, inv_t=1.25),
        # the gradient of a loss that the program forms from the log-probabilities itself
        dict(name="logp_grad_batch", op="logp_grad", rows=4096, vocab=32768, dtype="bf16", pad=0, inv_t=1.0),
        # one short response of a policy with a small vocabulary, loss and gradient
        dict(name="policy_short", op="policy", rows=63, vocab=32000, dtype="fp32", pad=0, kl=True, grad=True),
        # a microbatch of rollouts, loss with KL term and gradient
        dict(name="policy_batch", op="policy", rows=8192, vocab=131072, dtype="bf16", pad=0, kl=True, grad=True),
        # an odd vocabulary cut out of a wider buffer
        dict(name="policy_odd", op="policy", rows=2049, vocab=50021, dtype="fp16", pad=3, kl=False, grad=True),
        # one pair of short answers
        dict(name="preference_pair", op="preference", pairs=1, mean=40, split=1, vocab=32000, dtype="bf16", pad=0, grad=True),
        # a batch of pairs of ragged lengths, padded behind the last answer
        dict(name="preference_batch", op="preference", pairs=12, mean=200, split=2, vocab=131072, dtype="bf16", pad=0, grad=True),
        # the projections of two heads, where launches weigh most
        dict(name="orthogonal_heads", op="orthogonal", shapes="64x512,64x512", dtype="fp32", odtype="fp32"),
        # odd matrices of one list, tall and wide
        dict(name="orthogonal_odd", op="orthogonal", shapes="1000x777,513x2050,333x100,1025x1025", dtype="fp32", odtype="bf16"),
        # the step of a layer's attention weights
        dict(name="muon_attention", op="muon", shapes=f"{HIDDEN}x{HIDDEN},{KV}x{HIDDEN},{KV}x{HIDDEN},{HIDDEN}x{HIDDEN}",
             dtype="bf16", gdtype="bf16", master=False),
        # the step of a layer's two sides of the feed-forward product, binary32 masters
        dict(name="muon_ffn", op="muon", shapes=f"{FFN}x{HIDDEN},{HIDDEN}x{FFN}", dtype="bf16", gdtype="bf16", master=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp", "logp_grad", "policy", "policy", "preference", "preference", "orthogonal", "muon", "muon"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("logp", "logp_grad", "policy", "preference"):
        vocab = _log(rng, 1000, 200_000)
        if rng.random() < 0.6:
            vocab = vocab // 64 * 64
        most = min(16384, 500_000_000 // vocab)
        c = dict(op=op, vocab=vocab, dtype=dtype, pad=rng.choice([0, 0, 8, 3]))
        if op == "preference":
            c["pairs"] = _log(rng, 1, min(32, most // 32))
            c["mean"] = _log(rng, 12, max(13, min(1024, most // (2 * c["pairs"] + 1))))
            c["split"] = rng.randrange(1, 1 << 20)
            c["grad"] = rng.random() < 0.8
            return c
        c["rows"] = _log(rng, 1, most)
        if op == "policy":
            c["kl"], c["grad"] = rng.random() < 0.6, rng.random() < 0.8
        else:
            c["inv_t"] = rng.choice([1.0, 1.0, 0.75, 1.25])
        return c
    shapes, left = [], 60_000_000
    for _ in range(_log(rng, 1, 12)):
        rows, cols = _log(rng, 32, 4096), _log(rng, 32, 8192)
        if rng.random() < 0.5:
            rows, cols = cols // 32 * 32, rows // 32 * 32
        left -= rows * cols
        if left >= 0 or not shapes:
            shapes.append(f"{rows}x{cols}")
    c = dict(op=op, shapes=",".join(shapes), dtype=dtype)
    if op == "orthogonal":
        c["odtype"] = rng.choice([dtype, "fp32"])
    else:
        c["gdtype"] = rng.choice([dtype, "fp32"])
        c["master"] = dtype != "fp32" and rng.random() < 0.5
    return c


def shapes_of(case):
    return [tuple(int(k) for k in s.split("x")) for s in case["shapes"].split(",")]


def offsets_of(case):
    """First rows of the sequences of a preference batch (chosen ones first, then
    rejected ones) and one past the last; the batch has rows behind it."""
    r = random.Random(case["split"])
    at, offsets = 0, [0]
    for _ in range(2 * case["pairs"]):
        at += max(1, int(case["mean"] * r.uniform(0.4, 1.6)))
        offsets.append(at)
    return offsets, at + 5


def prompt_of(case, offsets):
    """Rows at the start of each sequence that belong to its prompt and take no part."""
    return [max(0, min(b - a - 1, (b - a) // 5)) for a, b in zip(offsets, offsets[1:])]


def rows_of(case):
    """Rows of the logits, rows that take part, rows whose gradient is written."""
    if case["op"] == "preference":
        offsets, rows = offsets_of(case)
        return rows, offsets[-1] - sum(prompt_of(case, offsets)), offsets[-1]
    rows = case["rows"]
    return rows, rows - len(range(15, rows, 16)), rows


# ---------------------------------------------------------------- what a program has in hand
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(n, scale):
        return torch.randn(n, generator=g, device="cuda") * scale

    def uniform(n, lo, hi):
        return torch.rand(n, generator=g, device="cuda") * (hi - lo) + lo

    s = {"case": case}
    if case["op"] in ("orthogonal", "muon"):
        shapes = shapes_of(case)
        s["rows"], s["cols"] = [a for a, _ in shapes], [b for _, b in shapes]
        s["coefs"] = [COEFS] * STEPS

        def update(a, b, size):
            # a gradient: noise, and a few directions that carry most of it
            k = min(16, a, b)
            x = normal((a, b), size)
            return x.addmm_(normal((a, k), 1.0) * torch.linspace(1, 0.1, k, device="cuda"), normal((k, b), size * 0.5))

        if case["op"] == "orthogonal":
            s["x"] = [update(a, b, 1e-3).to(DTYPES[case["dtype"]]) for a, b in shapes]
            s["y"] = [torch.empty((a, b), device="cuda", dtype=DTYPES[case["odtype"]]) for a, b in shapes]
            return s
        s["grads"] = [update(a, b, 1e-3).to(DTYPES[case["gdtype"]]) for a, b in shapes]
        s["momentum"] = [update(a, b, 6e-4) for a, b in shapes]
        w = [normal((a, b), 0.02) for a, b in shapes]
        s["params"] = [x.to(DTYPES[case["dtype"]]) for x in w]
        s["master"] = w if case["master"] else None
        s["scale"] = torch.full((1,), 0.25 + (seed % 8) / 16, device="cuda")
        return s

    vocab = case["vocab"]
    dt = DTYPES[case["dtype"]]
    rows, _, _ = rows_of(case)
    x = torch.empty((rows, vocab + case["pad"]), device="cuda", dtype=dt)
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    logp = torch.empty(rows, device="cuda")
    lse = torch.empty(rows, device="cuda")
    inv_t = case.get("inv_t", 1.0)
    part = max(1, 200_000_000 // vocab)
    for at in range(0, rows, part):
        # logits: a spread and a level of their own for each row, and the token that was sampled among the larger ones
        n = min(part, rows - at)
        z = normal((n, vocab + case["pad"]), 1.0) * uniform((n, 1), 1.0, 3.0) + normal((n, 1), 2.0)
        z.scatter_add_(1, targets[at:at + n, None], uniform((n, 1), 2.0, 14.0))
        x[at:at + n] = z.to(dt)
        z = x[at:at + n, :vocab].float() * inv_t
        top = z.amax(1, keepdim=True)
        t = z.gather(1, targets[at:at + n, None]) - top
        total = (z - top).exp_().sum(1, keepdim=True).log()
        logp[at:at + n] = (t - total).view(-1)
        lse[at:at + n] = (top + total).view(-1)
        del z
    s["logits"] = x[:, :vocab]
    if case["op"] != "preference":
        targets[15::16] = IGNORED  # a token in 16 was not sampled by the policy
    s["targets"], s["inv_t"] = targets, inv_t
    s["logp"] = torch.empty(rows, device="cuda")
    if case["op"] == "logp":
        s["lse"] = torch.empty(rows, device="cuda")
        return s
    s["dlogits"] = torch.zeros((rows, vocab), device="cuda", dtype=dt) if case.get("grad", True) else None
    if case["op"] == "logp_grad":
        s["lse"] = lse
        s["dlogp"] = normal(rows, 1.0)
        return s
    if case["op"] == "policy":
        # the policy has moved a little since the rollouts; no ratio lies on a border of the clipping
        d = normal(rows, 0.15)
        for border in (math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)):
            d = torch.where((d - border).abs() < 1e-3, d + 4e-3, d)
        s["old"] = logp - d
        s["ref"] = logp - normal(rows, 0.3) if case["kl"] else None
        s["advantage"] = normal(rows, 1.0) + 0.3
        s["weight"] = torch.full((rows,), 1.0 / rows, device="cuda")
        s["grad_scale"] = 1024.0 if case["dtype"] == "fp16" else 1.0
        s["token_loss"], s["loss"] = torch.empty(rows, device="cuda"), torch.empty(1, device="cuda")
        return s
    offsets, _ = offsets_of(case)
    prompt = prompt_of(case, offsets)
    for a, k in zip(offsets, prompt):
        targets[a:a + k] = IGNORED
    s["offsets"] = torch.tensor(offsets, device="cuda")
    sums = torch.stack([logp[a + k:b].sum() for a, b, k in zip(offsets, offsets[1:], prompt)])
    s["ref"] = sums + normal(2 * case["pairs"], 10.0)
    s["grad_scale"] = 1024.0 if case["dtype"] == "fp16" else 1.0
    s["logp"].zero_()
    s["seq_logp"], s["loss"] = torch.empty(2 * case["pairs"], device="cuda"), torch.empty(1, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def token_logp(s):
    """Log-probability of each row's target (0 where a row takes no part), the
    logarithm of the row's sum of exponentials, and the probabilities."""
    z = s["logits"].float() * s["inv_t"]
    counts = (s["targets"] >= 0) & (s["targets"] < z.shape[1])
    at = torch.where(counts, s["targets"], 0)[:, None]
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, at) - top
    e = z.sub_(top).exp_()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    logp = torch.where(counts, (picked - log_total).view(-1), 0.0)
    lse = torch.where(counts, (top + log_total).view(-1), 0.0)
    return logp, lse, e, total, counts, at


def logits_grad(s, dlogp, p, counts, at):
    """dlogp * d logp / d logits, from the probabilities p (overwritten)."""
    d = (dlogp * s["inv_t"])[:, None]
    dz = p.neg_().scatter_add_(1, at, torch.ones_like(d)).mul_(d)
    return torch.where(counts[:, None], dz, 0.0).to(s["logits"].dtype)


def _plain_logp(s):
    logp, lse, *_ = token_logp(s)
    return logp, lse


def _plain_logp_grad(s):
    counts = (s["targets"] >= 0) & (s["targets"] < s["logits"].shape[1])
    at = torch.where(counts, s["targets"], 0)[:, None]
    p = (s["logits"].float() * s["inv_t"]).sub_(s["lse"][:, None]).exp_()
    return logits_grad(s, s["dlogp"], p, counts, at)


def _plain_policy(s):
    logp, _, e, total, counts, at = token_logp(s)
    w = torch.where(counts, s["weight"], 0.0)
    ratio = torch.exp(logp - s["old"])
    a = s["advantage"]
    free, held = ratio * a, torch.clamp(ratio, 1 - CLIP_LOW, 1 + CLIP_HIGH) * a
    token = -torch.minimum(free, held)
    dlogp = torch.where(free <= held, -free, 0.0)
    if s["ref"] is not None:
        back = torch.exp(s["ref"] - logp)
        token = token + KL * (back - (s["ref"] - logp) - 1)
        dlogp = dlogp + KL * (1 - back)
    token = torch.where(counts, token * w, 0.0)
    loss = token.double().sum().float().view(1)
    out = [loss, token, logp]
    if s["dlogits"] is not None:
        out.append(logits_grad(s, dlogp * w * s["grad_scale"], e.div_(total), counts, at))
    return out


def _plain_preference(s):
    n, pairs = s["offsets"], s["case"]["pairs"]
    logp, _, e, total, counts, at = token_logp(s)
    row = torch.arange(logp.numel(), device="cuda")
    seq = torch.searchsorted(n, row, right=True) - 1              # each row's sequence
    inside = (seq >= 0) & (seq < 2 * pairs)
    seq = torch.where(inside, seq, 0)
    counts = counts & inside
    logp = torch.where(counts, logp, 0.0)
    sums = torch.zeros(2 * pairs, device="cuda", dtype=torch.float64).index_add_(0, seq, logp.double())
    h = BETA * ((sums[:pairs] - s["ref"][:pairs].double()) - (sums[pairs:] - s["ref"][pairs:].double()))
    soft = lambda x: torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))  # noqa: E731  log(1 + exp(x))
    loss = ((1 - SMOOTHING) * soft(-h) + SMOOTHING * soft(h)).mean().float().view(1)
    s["logp"].copy_(torch.where(inside, logp, s["logp"]))
    out = [loss, sums.float(), s["logp"]]
    if s["dlogits"] is not None:
        up = 1 / (1 + torch.exp(-h))
        dh = (SMOOTHING * up - (1 - SMOOTHING) * (1 - up)) * (BETA / pairs * s["grad_scale"])
        dz = logits_grad(s, torch.cat([dh, -dh]).float()[seq], e.div_(total), counts, at)
        out.append(torch.where(inside[:, None], dz, s["dlogits"]))
    return out


def orthogonalized(x):
    """Newton-Schulz products on one binary32 matrix."""
    a, b, c = COEFS
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (torch.sqrt((x.double() * x.double()).sum()).float() + NORM_EPS)
    for _ in range(STEPS):
        m = x @ x.t()
        x = a * x + (b * m + c * (m @ m)) @ x
    return x.t() if tall else x


def _plain_orthogonal(s):
    return [orthogonalized(x.float()).to(y.dtype).contiguous() for x, y in zip(s["x"], s["y"])]


def _plain_muon(s):
    for i, (p, g, m) in enumerate(zip(s["params"], s["grads"], s["momentum"])):
        g = g.float() * s["scale"]
        m.copy_(MOMENTUM * m + (1 - MOMENTUM) * g)
        o = orthogonalized((1 - MOMENTUM) * g + MOMENTUM * m)
        w = s["master"][i] if s["master"] else p
        new = (1 - LR * DECAY) * w.float() - LR * math.sqrt(max(1.0, p.shape[0] / p.shape[1])) * o
        if s["master"]:
            w.copy_(new)
        p.copy_(new)
    return [s["params"], s["momentum"]] + ([s["master"]] if s["master"] else [])


# ---------------------------------------------------------------- the package's operators
def _own_logp(s):
    import allgather_rr_allreduce_gb300 as rr
    x = s["logits"]
    rr.rr_token_logp(x, s["targets"], s["logp"], s["lse"], x.shape[0], x.shape[1], x.stride(0), s["inv_t"],
                     s["case"]["dtype"])
    return s["logp"], s["lse"]


def _own_logp_grad(s):
    import allgather_rr_allreduce_gb300 as rr
    x, d = s["logits"], s["dlogits"]
    rr.rr_token_logp_backward(x, s["targets"], s["lse"], s["dlogp"], d, x.shape[0], x.shape[1], x.stride(0),
                              d.stride(0), s["inv_t"], s["case"]["dtype"])
    return d


def _own_policy(s):
    import allgather_rr_allreduce_gb300 as rr
    x, d = s["logits"], s["dlogits"]
    hyper = rr.rr_policy_hyper(CLIP_LOW, CLIP_HIGH, KL, s["inv_t"], s["grad_scale"])
    rr.rr_policy_loss(x, s["targets"], s["old"], s["ref"], s["advantage"], s["weight"], s["loss"], s["token_loss"],
                      s["logp"], d, x.shape[0], x.shape[1], x.stride(0), 0 if d is None else d.stride(0), hyper,
                      s["case"]["dtype"])
    return [s["loss"], s["token_loss"], s["logp"]] + ([] if d is None else [d])


def _own_preference(s):
    import allgather_rr_allreduce_gb300 as rr
    x, d, pairs = s["logits"], s["dlogits"], s["case"]["pairs"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(rr.rr_preference_loss_workspace(x.shape[0], pairs), device="cuda", dtype=torch.uint8)
    hyper = rr.rr_preference_hyper(BETA, SMOOTHING, 0.0, s["inv_t"], s["grad_scale"], 0)
    rr.rr_preference_loss(x, s["targets"], s["offsets"], s["ref"], s["loss"], s["seq_logp"], s["logp"], d, x.shape[0],
                          x.shape[1], x.stride(0), 0 if d is None else d.stride(0), pairs, hyper, s["case"]["dtype"],
                          s["workspace"], s["workspace"].numel())
    return [s["loss"], s["seq_logp"], s["logp"]] + ([] if d is None else [d])


def _own_orthogonal(s):
    import allgather_rr_allreduce_gb300 as rr
    if "workspace" not in s:
        s["workspace"] = torch.empty(rr.rr_orthogonalize_workspace(s["rows"], s["cols"]), device="cuda", dtype=torch.uint8)
    rr.rr_orthogonalize(s["x"], s["y"], s["rows"], s["cols"], s["case"]["dtype"], s["case"]["odtype"], s["coefs"],
                        NORM_EPS, s["workspace"], s["workspace"].numel())
    return s["y"]


def _own_muon(s):
    import allgather_rr_allreduce_gb300 as rr
    if "workspace" not in s:
        s["workspace"] = torch.empty(rr.rr_orthogonalize_workspace(s["rows"], s["cols"]), device="cuda", dtype=torch.uint8)
    hyper = rr.rr_muon_hyper(LR, MOMENTUM, DECAY, NORM_EPS, 1, rr.RR_MUON_SPECTRAL)
    rr.rr_muon(s["params"], s["grads"], s["momentum"], s["master"], s["rows"], s["cols"], s["case"]["dtype"],
               s["case"]["gdtype"], hyper, s["coefs"], s["scale"], s["workspace"], s["workspace"].numel())
    return [s["params"], s["momentum"]] + ([s["master"]] if s["master"] else [])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"logp": _own_logp, "logp_grad": _own_logp_grad, "policy": _own_policy, "preference": _own_preference,
                "orthogonal": _own_orthogonal, "muon": _own_muon}[op](state)
    return {"logp": _plain_logp, "logp_grad": _plain_logp_grad, "policy": _plain_policy, "preference": _plain_preference,
            "orthogonal": _plain_orthogonal, "muon": _plain_muon}[op](state)


# ---------------------------------------------------------------- work and exact values
def work(case):
    op = case["op"]
    if op in ("orthogonal", "muon"):
        shapes = [(min(a, b), max(a, b)) for a, b in shapes_of(case)]
        n = sum(a * b for a, b in shapes)
        # of a symmetric product only a half: X X' and its square, then their sum times X
        flops = STEPS * sum(m * m * k + m * m * m + 2 * m * m * k for m, k in shapes)
        if op == "orthogonal":
            return {"bytes": n * (BYTES[case["dtype"]] + BYTES[case["odtype"]]), "flops": flops}
        each = BYTES[case["gdtype"]] + 8 + (8 + BYTES[case["dtype"]] if case["master"] else 2 * BYTES[case["dtype"]])
        return {"bytes": n * each, "flops": flops + 10 * n}
    rows, counted, written = rows_of(case)
    b, vocab = BYTES[case["dtype"]], case["vocab"]
    if op == "logp":
        return {"bytes": counted * vocab * b + rows * 16, "flops": 4 * counted * vocab}
    if op == "logp_grad":
        return {"bytes": (counted + written) * vocab * b + rows * 16, "flops": 4 * counted * vocab}
    moved = counted + (written if case["grad"] else 0)
    return {"bytes": moved * vocab * b + rows * 28, "flops": (8 if case["grad"] else 4) * counted * vocab}


def _exact_orthogonal(x, coefs):
    """Every product of the iteration is a polynomial in X X' times X, so the
    polynomial is built up on the short side and X is multiplied once."""
    tall = x.shape[0] > x.shape[1]
    x = x.mT if tall else x
    x = x / (torch.linalg.matrix_norm(x) + NORM_EPS)
    gram = torch.einsum("ik,jk->ij", x, x)
    total = None
    for a, b, c in coefs:
        p = torch.mm(gram, gram).mul_(c).add_(gram, alpha=b)
        p.diagonal().add_(a)
        total = p if total is None else p @ total
        gram = p @ gram @ p
    x = total @ x
    return x.mT.contiguous() if tall else x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "orthogonal":
        return [_exact_orthogonal(x.double(), s["coefs"]) for x in s["x"]]
    if op == "muon":
        params, moments = [], []
        for i, (a, b) in enumerate(shapes_of(case)):
            g = s["grads"][i].double() * s["scale"].double()
            m = torch.lerp(g, s["momentum"][i].double(), MOMENTUM)
            o = _exact_orthogonal(torch.lerp(g, m, MOMENTUM), s["coefs"])
            w = (s["master"] if s["master"] else s["params"])[i].double()
            params.append(w - LR * DECAY * w - LR * max(1.0, a / b) ** 0.5 * o)
            moments.append(m)
        return [params, moments] + ([params] if s["master"] else [])
    z = s["logits"].double() * s["inv_t"]
    targets, vocab = s["targets"], case["vocab"]
    rows = torch.nonzero((targets >= 0) & (targets < vocab)).view(-1)
    if op == "preference":
        rows = rows[rows < offsets_of(case)[0][-1]]
    picked = targets[rows]
    p = torch.log_softmax(z, 1)
    logp = torch.zeros(z.shape[0], device="cuda", dtype=torch.float64)
    logp[rows] = p[rows, picked]
    if op == "logp":
        lse = torch.zeros_like(logp)
        lse[rows] = z[rows, picked] - logp[rows]
        return logp, lse
    p.exp_()
    del z

    def grad(d):
        """d * (one at the target - probabilities), zeros in the other rows."""
        dz = torch.zeros_like(p)
        dz[rows] = p[rows] * -d[rows, None]
        dz[rows, picked] += d[rows]
        return dz

    if op == "logp_grad":
        return grad(s["dlogp"].double() * s["inv_t"])
    if op == "policy":
        ratio, a = (logp - s["old"].double()).exp(), s["advantage"].double()
        low, high = 1 - CLIP_LOW, 1 + CLIP_HIGH
        clipped = ((a > 0) & (ratio > high)) | ((a < 0) & (ratio < low))
        token = -a * torch.where(clipped, ratio.clamp(low, high), ratio)
        slope = torch.where(clipped, 0.0, -a * ratio)
        if case["kl"]:
            gap = s["ref"].double() - logp
            token += KL * (torch.expm1(gap) - gap)
            slope -= KL * torch.expm1(gap)
        weight = torch.zeros_like(logp)
        weight[rows] = s["weight"][rows].double()
        token, slope = token * weight, slope * weight
        out = [token.sum().view(1), token, logp]
        return out + ([grad(slope * s["grad_scale"])] if case["grad"] else [])
    pairs, (offsets, _) = case["pairs"], offsets_of(case)
    sums = torch.stack([logp[a:b].sum() for a, b in zip(offsets, offsets[1:])])
    margin = (sums - s["ref"].double()).view(2, pairs)
    h = BETA * (margin[0] - margin[1])
    logsig = torch.nn.functional.logsigmoid
    loss = -((1 - SMOOTHING) * logsig(h) + SMOOTHING * logsig(-h)).mean().view(1)
    out = [loss, sums, logp]
    if case["grad"]:
        slope = (torch.sigmoid(h) - (1 - SMOOTHING)) * BETA / pairs * s["grad_scale"]
        d = torch.zeros_like(logp)
        for k, v in enumerate([*slope, *-slope]):
            d[offsets[k]:offsets[k + 1]] = v
        out.append(grad(d))
    return out
