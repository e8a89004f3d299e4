"""Factors of 0 of the policy loss (an advantage, a weight, the KL term's
coefficient, the gradient's scale) leave out what they multiply, also where that
is more than binary32 holds.  In 64 bits it is finite, and the product 0."""
import math

import pytest
import torch

from logits_util import Reference, make
from step_util import U24 as u, within

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")
INF = math.inf


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


def call(rr, x, t, old, ref, adv, weight, hyper):
    rows, vocab = x.shape
    token, lp = torch.empty((2, rows), **CUDA)
    loss, dx = torch.empty(1, **CUDA), torch.empty_like(x)
    rr.rr_policy_loss(x, t, old, ref, adv, weight, loss, token, lp, dx, rows, vocab, vocab, vocab,
                      rr.rr_policy_hyper(*hyper), "fp32")
    return loss, token, dx


def columns(*rows):
    return list(torch.tensor(rows, dtype=torch.float32, **CUDA).t().contiguous())


@pytest.mark.parametrize("vocab", [50, 40000])
def test_zero_advantages_and_weights(rr, vocab):
    # old, ref, advantage, weight; log-probabilities are near -10, so ratios of old -200 and KL terms of ref +200 overflow
    old, ref, adv, weight = columns((-200, -10, 0, 1), (-200, -10, -1, 0), (-10, 200, 1, 0), (-200, 200, -2, 0), (-200, -10, 0, 0))
    x, t, _ = make(5, vocab, "fp32", seed=1, ignored=0)
    want = Reference(x, t, 1.0)
    for high in (0.2, INF):
        loss, token, dx = call(rr, x, t, old, ref, adv, weight, (0.2, high, 0.1, 1.0, 1.0))
        gap = float(ref[0]) - float(want.logp[0])
        kl = 0.1 * (math.expm1(gap) - gap)
        assert bool((token[1:] == 0).all()) and bool((dx[1:] == 0).all())
        # the first row's KL term is all of the loss
        room = 0.1 * (abs(math.expm1(gap)) * float(want.logp_tol[0]) + 6 * u * (abs(math.expm1(gap)) + abs(gap))) + 4 * u * kl
        assert abs(float(token[0]) - kl) <= room and float(loss) == float(token[0])
        assert bool(torch.isfinite(dx[0]).all())


@pytest.mark.parametrize("vocab", [50, 40000])
def test_zero_coefficient_leaves_the_term_out(rr, vocab):
    x, t, g = make(6, vocab, "fp32", seed=2, ignored=0)
    x[5, t[5]] = -INF  # a masked target
    lp = torch.log_softmax(x.double(), 1).gather(1, t[:, None]).view(-1)
    old = torch.where(torch.isfinite(lp), lp, -3.0).float() - 0.05
    ref = torch.full((6,), 150.0, **CUDA)
    adv = torch.randn(6, generator=g, **CUDA)
    with_ref = call(rr, x, t, old, ref, adv, None, (0.2, 0.2, 0.0, 1.0, 1.0))
    without = call(rr, x, t, old, None, adv, None, (0.2, 0.2, 0.0, 1.0, 1.0))
    for a, b in zip(with_ref, without):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


@pytest.mark.parametrize("vocab", [50, 40000])
def test_opposite_infinities(rr, vocab):
    """The policy's and the KL term's parts overflow to both sides: gains without a clip, slopes of a negative advantage."""
    x, t, _ = make(2, vocab, "fp32", seed=6, ignored=0)
    old, ref, adv, weight = columns((-200, 200, 2, 0), (-200, 200, -2, 0))
    loss, token, dx = call(rr, x, t, old, ref, adv, weight, (0.2, INF, 0.1, 1.0, 1.0))
    assert bool((token == 0).all()) and float(loss) == 0 and bool((dx == 0).all())
    _, _, dx = call(rr, x, t, old, ref, adv, None, (0.2, INF, 0.1, 1.0, 0.0))
    assert bool((dx == 0).all())


def test_zero_gradient_scale(rr):
    x, t, _ = make(3, 50, "fp32", seed=3, ignored=0)
    old, adv = torch.full((3,), -200.0, **CUDA), torch.full((3,), -1.0, **CUDA)
    loss, token, dx = call(rr, x, t, old, None, adv, None, (0.2, 0.2, 0.0, 1.0, 0.0))
    assert bool((token == INF).all()) and float(loss) == INF and bool((dx == 0).all())


@pytest.mark.parametrize("vocab", [50, 40000])
def test_masked_target_costs_infinitely_much(rr, vocab):
    """exp(gap) - gap - 1 of a gap that is +inf, not a difference of two infinities."""
    x, t, _ = make(2, vocab, "fp32", seed=5, ignored=0)
    x[0, t[0]] = -INF
    old, ref, adv = columns((-3, -2, 1), (-3, -2, 1))
    loss, token, _ = call(rr, x, t, old, ref, adv, None, (0.2, 0.2, 0.1, 1.0, 1.0))
    assert float(token[0]) == INF and math.isfinite(float(token[1])) and float(loss) == INF


def test_what_stays(rr):
    """Infinite losses stay infinite, NaN stays NaN, ordinary rows beside them are untouched."""
    x, t, _ = make(4, 1000, "fp32", seed=4, ignored=0)
    ref = Reference(x, t, 1.0)
    old = torch.stack([torch.tensor(-200.0, **CUDA), torch.tensor(math.nan, **CUDA), ref.logp[2].float(), ref.logp[3].float()])
    adv, weight = columns((-1, 1), (1, 0), (1, 1), (-1, 0.5))
    loss, token, dx = call(rr, x, t, old, None, adv, weight, (0.2, 0.2, 0.0, 1.0, 1.0))
    assert float(token[0]) == INF and math.isnan(float(token[1])) and math.isnan(float(loss))
    assert bool(torch.isnan(dx[1]).all())
    slope = torch.tensor([0.0, 0.0, -1.0, 0.5], **CUDA).double()
    want, tol = ref.grad(slope, slope.abs() * (ref.logp_tol + 8 * u * (1 + ref.logp.abs())), "fp32")
    within(dx[2:], want[2:], tol[2:], "dlogits")
