"""A preference loss whose sequences hold masked targets (-inf logits): a term of
the loss whose weight is 0 stays out of it, also where it is infinite."""
import math

import pytest
import torch

from logits_util import Reference, make
from step_util import U24 as u, within

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")
OFFSETS = [0, 3, 7, 9, 12, 16, 20]  # three pairs


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


@pytest.mark.parametrize("smoothing,masked,infinite", [(0.0, "rejected", False), (1.0, "chosen", False), (0.1, "rejected", True),
                                                       (0.0, "chosen", True)])
@pytest.mark.parametrize("average", [0, 1])
def test_masked_targets(rr, smoothing, masked, infinite, average):
    rows, vocab, pairs = 20, 301, 3
    x, t, _ = make(rows, vocab, "fp32", seed=2, ignored=0)
    seq_of = 1 if masked == "chosen" else 4  # of the second pair
    x[OFFSETS[seq_of], t[OFFSETS[seq_of]]] = -math.inf
    ref = Reference(x, t, 1.0)
    hyper = rr.rr_preference_hyper(0.3, smoothing, 0.1, 1.0, 1.0, average)
    loss, seq, lp, dx = torch.empty(1, **CUDA), torch.empty(6, **CUDA), torch.empty(rows, **CUDA), torch.empty_like(x)
    space = torch.empty(rr.rr_preference_loss_workspace(rows, pairs), **CUDA, dtype=torch.uint8)
    rr.rr_preference_loss(x, t, torch.tensor(OFFSETS, **CUDA), None, loss, seq, lp, dx, rows, vocab, vocab, vocab, pairs, hyper,
                          "fp32", space, space.numel())
    assert float(seq[seq_of]) == -math.inf
    total, total_tol = 0.0, 0.0
    slope, slope_tol = torch.zeros(rows, **CUDA).double(), torch.zeros(rows, **CUDA).double()
    beta, margin, eps = (float(torch.tensor(v, dtype=torch.float32)) for v in (0.3, 0.1, smoothing))
    for p in range(pairs):
        parts = [slice(OFFSETS[q], OFFSETS[q + 1]) for q in (p, p + pairs)]
        n = [(s.stop - s.start) if average else 1 for s in parts]
        s = [float(ref.logp[k].sum()) / m for k, m in zip(parts, n)]
        h = beta * (s[0] - s[1]) - margin
        finite = math.isfinite(h)
        # sums, their difference and h round once each; slopes of softplus and of its derivative are below 1
        h_tol = beta * sum(float(ref.logp_tol[k].sum()) / m for k, m in zip(parts, n)) + 3 * u * abs(h) if finite else 0.0
        soft = lambda v: max(v, 0.0) + math.log1p(math.exp(-abs(v)))  # noqa: E731
        for w, v in ((1 - eps, -h), (eps, h)):
            if w > 0:
                total += w * soft(v) / pairs
                total_tol += (w * (h_tol + 12 * u * soft(v)) if finite else 0.0) / pairs
        sig = (1 / (1 + math.exp(-h)) if h > -700 else 0.0) if finite else float(h > 0)
        dh = (eps * sig - (1 - eps) * (1 - sig)) * beta / pairs
        for k, m, sign in zip(parts, n, (1, -1)):
            slope[k] = sign * dh / m
            slope_tol[k] = (h_tol * 0.25 + 16 * u) * beta / pairs / m if finite else 4 * u * abs(dh) / m
    if infinite:
        assert float(loss) == math.inf and total == math.inf
    else:
        assert abs(float(loss) - total) <= total_tol + 3 * u * total, (float(loss), total)
    want, tol = ref.grad(slope, slope_tol, "fp32")
    # a masked place has probability 0, and its bound is the target's alone
    tol = torch.where(torch.isfinite(tol), tol, 2 * u * slope.abs()[:, None] + slope_tol[:, None])
    within(dx, want, tol, "dlogits")
