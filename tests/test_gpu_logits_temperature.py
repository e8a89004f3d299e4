"""Log-probabilities and their gradient at the ends of the temperature's range."""
import pytest
import torch

from logits_util import Reference, make
from step_util import U24 as u, within

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")


@pytest.mark.parametrize("inv_t", [2.0 ** -120, 2.0 ** -40, 2.0 ** 40, 2.0 ** 120])
@pytest.mark.parametrize("rows,vocab", [(5, 100), (2, 40000)])
def test_ends_of_the_range(rows, vocab, inv_t):
    import allgather_rr_allreduce_gb300 as rr
    x, t, g = make(rows, vocab, "fp32", seed=vocab, ignored=0)
    ref = Reference(x, t, inv_t)
    logp, lse = torch.empty((2, rows), **CUDA)
    rr.rr_token_logp(x, t, logp, lse, rows, vocab, vocab, inv_t, "fp32")
    within(logp, ref.logp, ref.logp_tol, "logp")
    within(lse, ref.lse, ref.lse_tol, "lse")
    d, dx = torch.randn(rows, generator=g, **CUDA), torch.empty_like(x)
    rr.rr_token_logp_backward(x, t, lse, d, dx, rows, vocab, vocab, vocab, inv_t, "fp32")
    # the base lse / inv_t and the difference from it round at the size of the logits
    extra = u * 6 * (ref.lse.abs() + ref.z.abs().amax(1)) + ref.lse_tol
    want, tol = ref.grad(d.double(), torch.zeros_like(ref.lse), "fp32", extra)
    if inv_t < 1:  # at 2^40 and more a probability turns on lse's last bit: the bound holds nothing then
        within(dx, want, tol, "dlogits")
    else:
        assert not bool(torch.isnan(dx).any())
