"""rr_adamw8 bit for bit where its fast roots and quotients may not be used:
averages near binary32's smallest and largest values beside ordinary ones,
quotients that overflow or leave the normal range, exact zeros.  Weights are
zero, so that what a step adds to them is the whole result."""
import numpy as np
import pytest
import torch

from step_util import generator
from test_gpu_adamw import H, check_adamw8, lists8, rr, run_adamw8, snapshot8  # noqa: F401

pytestmark = pytest.mark.gpu


def states(n, seed, mscale, rscale, least_code=0, gdtype="fp32", shift=0):
    """Random codes of at least `least_code` under the two scales, no gradient, weights of zero."""
    L = lists8([n], [shift], seed, "fp32", gdtype, False)
    for name, scale in (("m", mscale), ("r", rscale)):
        L[name + "s"][0].t.fill_(scale)
        code = torch.randint(least_code, 0x7F, (n,), generator=generator(seed + len(name)), device="cuda")
        if name == "m":
            code = code + 128 * torch.randint(0, 2, (n,), generator=generator(seed + 9), device="cuda")
        L[name][0].t.copy_(code)
    L["g"][0].t.zero_()
    L["p"][0].t.zero_()
    return L


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("name,mscale,rscale,least,h", [
    ("m near the smallest normal value", 2.0 ** -126, 2.0 ** -20, 0, {}),
    ("m a little above it", 2.0 ** -118, 2.0 ** -24, 0x38, dict(eps=0.0)),
    ("m above that", 2.0 ** -110, 2.0 ** -30, 0, dict(eps=1e-12)),
    ("m of 2^100 over roots of 2^-50", 2.0 ** 91, 2.0 ** -49, 0x40, dict(eps=0.0)),
    ("m of 2^90 over roots of 2^-40", 2.0 ** 81, 2.0 ** -41, 0x40, dict(eps=0.0)),
    ("a quotient below the normal range", 2.0 ** -92, 2.0 ** 40, 0x38, {}),
    ("a large eps", 2.0 ** -90, 2.0 ** -10, 0x38, dict(eps=2.0 ** 45)),
    ("a beta1 that takes the scale below the normal range", 2.0 ** -60, 2.0 ** -30, 0x38, dict(beta1=1e-25)),
    ("a small quotient after one step", 2.0 ** -95, 2.0 ** 18, 0, dict(step=1, beta2=0.999999)),
    ("ordinary values", 2.0 ** -20, 2.0 ** -20, 0, {}),
    ("no decay at all", 2.0 ** -125, 2.0 ** -20, 0, dict(beta1=0.0)),
])
def test_far_states_bit_for_bit(rr, name, mscale, rscale, least, h, shift):  # noqa: F811
    n = 5003
    L = states(n, 30, mscale, rscale, least, shift=shift)
    old = snapshot8(L)
    run_adamw8(rr, L, [n], "fp32", "fp32", None, **h)
    check_adamw8(L, old, [n], "fp32", 1.0, 12345, {**H, **h})
    if least:
        assert bool((L["p"][0].t != 0).any()) or h.get("beta1") == 1e-25


def test_zeros_among_ordinary_averages(rr):  # noqa: F811
    """Averages that are exactly zero (either sign) beside ordinary ones, in every
    lane's place, with and without weights to move."""
    n = 4096
    for weight in (0.0, 0.05):
        L = states(n, 31, 2.0 ** -20, 2.0 ** -20, 0x38)
        L["p"][0].t.fill_(weight)
        m = L["m"][0].t
        m[::7] = 0
        m[3::11] = 0x80
        old = snapshot8(L)
        run_adamw8(rr, L, [n], "fp32", "fp32")
        check_adamw8(L, old, [n], "fp32", 1.0, 12345, H)


def test_scales_from_the_smallest_to_the_largest(rr):  # noqa: F811
    """A block for each pair of scales, four binades apart."""
    exps = np.arange(-126, 121, 13)
    pairs = [(a, b) for a in exps for b in exps if b <= 60]
    n = 256 * len(pairs)
    L = states(n, 32, 1.0, 1.0)
    for k, name in ((0, "ms"), (1, "rs")):
        L[name][0].t.copy_(torch.tensor([2.0 ** int(p[k]) for p in pairs]))
    for h in ({}, dict(eps=0.0), dict(eps=1e-20, beta1=0.5, step=1)):
        old = snapshot8(L)
        run_adamw8(rr, L, [n], "fp32", "fp32", None, **h)
        check_adamw8(L, old, [n], "fp32", 1.0, 12345, {**H, **h})
        L["p"][0].t.zero_()


def test_codes_that_overflow_under_their_scale(rr):  # noqa: F811
    """256 and more times 2^120 is infinite: the block is, whatever beta1."""
    n = 1024
    L = states(n, 33, 2.0 ** 120, 2.0 ** -20, 0x38)
    L["m"][0].t[256:] = 0x40     # blocks whose values are finite
    old = snapshot8(L)
    run_adamw8(rr, L, [n], "fp32", "fp32")
    check_adamw8(L, old, [n], "fp32", 1.0, 12345, H)
    assert np.isnan(L["ms"][0].t.cpu().numpy()).tolist() == [True, False, False, False]
