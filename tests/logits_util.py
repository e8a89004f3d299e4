"""The losses over logits in 64 bits, and how far binary32 may be from them.

Bounds (u = 2^-24).  A term exp(z_j - max) has its exponent rounded three times
(difference, factor, product): relative 3u |z_j - max|, and ex2.approx adds 4u.
A thread rescales its sum whenever its maximum moves, and the joins of threads,
warps and blocks do so 15 times more: at most `chunks + 16` factors of 4u each.
A thread of 256 adds vocab / 512 terms to each of two sums (a warp's lanes and the
blocks' join: 16 more): u each.  What the sum is off by, relative, is what its
logarithm is off by, and logf and the differences around it add a few u."""
import torch

from step_util import TORCH, U, U24 as u

ROW_FACTORS = 16


def make(rows, vocab, dtype, seed, pad=0, shift=0, ignored=0.2, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = vocab + pad
    flat = torch.empty(rows * wide + shift, device="cuda", dtype=TORCH[dtype])
    flat.copy_(torch.randn(flat.numel(), generator=g, device="cuda") * spread)
    x = flat[shift:].view(rows, wide)[:, :vocab]
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    skip = torch.rand(rows, generator=g, device="cuda") < ignored
    t = torch.where(skip, torch.where(torch.arange(rows, device="cuda") % 2 == 0, -100, vocab), t)
    return x, t, g


class Reference:
    """Row statistics in 64 bits and their tolerances."""

    def __init__(self, x, target, inv_t):
        self.vocab = x.shape[1]
        self.counts = (target >= 0) & (target < self.vocab)
        self.at = torch.where(self.counts, target, 0)[:, None]
        inv_t = float(torch.tensor(inv_t, dtype=torch.float32))
        self.inv_t = inv_t
        self.z = x.double() * inv_t
        top = self.z.amax(1, keepdim=True)
        e = (self.z - top).exp()
        total = e.sum(1, keepdim=True)
        self.p = e / total
        gap = (top - self.z)
        self.lse = torch.where(self.counts, (top + total.log()).view(-1), 0.0)
        picked = (self.z.gather(1, self.at) - top).view(-1)
        self.logp = torch.where(self.counts, picked - total.log().view(-1), 0.0)
        per = 16 // x.element_size()
        factors = -(-self.vocab // (256 * per * 4)) + ROW_FACTORS
        first = torch.where(self.p > 0, self.p * gap, 0.0).sum(1)
        self.sum_tol = u * (4 * (factors + 1) + 3 * first + self.vocab / 512 + 16)
        log_total = total.log().view(-1).abs()
        self.logp_tol = self.sum_tol + u * (2 * log_total + 3 * picked.abs() + 2 * self.logp.abs()) + u
        self.lse_tol = self.sum_tol + u * (2 * log_total + 3 * top.view(-1).abs() + 2 * self.lse.abs()) + u
        # relative error of a probability: its term, the sum (or lse), quotient and product
        self.p_tol = self.sum_tol[:, None] + u * (8 + 3 * gap)

    def grad(self, slope, slope_tol, dtype, extra=None):
        """d * inv_t * (1[target] - p) with its tolerance, zeros where a row takes no part; `extra`: relative
        error that the base of the exponents brings."""
        slope = torch.where(self.counts, slope, 0.0) * self.inv_t
        tol = slope_tol * self.inv_t + 2 * u * slope.abs()
        one = torch.zeros_like(self.p).scatter_(1, self.at, 1.0)
        want = torch.where(self.counts[:, None], slope[:, None] * (one - self.p), 0.0)
        rel = self.p_tol + (0 if extra is None else extra[:, None])
        off = slope.abs()[:, None] * (self.p * rel + one * 2 * u) + tol[:, None] * (one + self.p)
        off = off + U[dtype] * (want.abs() + off) + {"bf16": 2.0 ** -126, "fp16": 2.0 ** -25, "fp32": 2.0 ** -126}[dtype]
        return want, torch.where(self.counts[:, None], off, 0.0)


def policy(ref, old, kl_ref, adv, weight, hyper):
    """token losses and slopes with their tolerances; weight and old may be None."""
    low, high = 1 - hyper.clip_low, 1 + hyper.clip_high
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    low, high, kl = f32(low), f32(high), f32(hyper.kl_coef)
    one = torch.ones_like(ref.logp)
    w = one if weight is None else weight.double()
    a = adv.double()
    diff = torch.zeros_like(ref.logp) if old is None else ref.logp - old.double()
    ratio = diff.exp()
    ratio_tol = torch.zeros_like(ratio) if old is None else ratio * (ref.logp_tol + u * diff.abs() + 4 * u)
    free, held = ratio * a, ratio.clamp(low, high) * a
    token = -torch.minimum(free, held)
    slope = torch.where(free <= held, -free, 0.0)
    tol = a.abs() * ratio_tol + 2 * u * free.abs()
    token_tol, slope_tol = tol.clone(), tol.clone()
    if kl_ref is not None:
        gap = kl_ref.double() - ref.logp
        back = torch.expm1(gap)
        gap_tol = ref.logp_tol + u * gap.abs()
        back_tol = gap.exp() * gap_tol + 4 * u * back.abs()
        token = token + kl * (back - gap)
        slope = slope - kl * back
        # (back - gap) moves with the gap as back does; its difference rounds once
        token_tol = token_tol + kl * (back.abs() * gap_tol + 4 * u * back.abs() + u * gap.abs() * 2) + 3 * u * token.abs()
        slope_tol = slope_tol + kl * back_tol + 3 * u * slope.abs()
    zero = torch.zeros_like(token)
    token = torch.where(ref.counts, token * w, zero)
    return (token, torch.where(ref.counts, token_tol * w.abs() + u * token.abs(), zero),
            slope * w, slope_tol * w.abs() + 2 * u * (slope * w).abs())
