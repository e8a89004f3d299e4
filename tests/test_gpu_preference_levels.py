"""The preference loss's gradient does not lose exactness where logits lie far
from zero: its probabilities come from differences to the row's maximum, so the
bound has no term of the logits' size."""
import pytest
import torch

from logits_util import Reference
from test_gpu_logits import guarded_rows, pair_case, preference
from step_util import within

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("level", [0.0, 15.0, 100.0, 1000.0, -1000.0, 20000.0])
@pytest.mark.parametrize("lens,vocab", [((20, 30), 32000), ((17, 3, 0, 9, 1, 40), 1025), ((2, 1), 131072)])
def test_gradient_at_levels(rr, lens, vocab, level, dtype):
    for pad, shift, inv_t in ((0, 0, 1.0), (3, 1, 0.75)):
        x, t, offsets, g = pair_case(lens, vocab, dtype, seed=vocab, pad=pad, shift=shift)
        x.copy_(x.float() + level)
        rows, pairs = x.shape[0], len(lens) // 2
        ref = Reference(x, t, inv_t)
        sums = torch.stack([ref.logp[a:b].sum() for a, b in zip(offsets.tolist(), offsets.tolist()[1:])])
        seq_ref = (sums + torch.randn(len(lens), generator=g, **CUDA) * 8).float()
        hyper = rr.rr_preference_hyper(0.1, 0.1, 0.0, inv_t, 256.0, 0)
        loss, seq, lp = torch.empty(1, **CUDA), torch.empty(2 * pairs, **CUDA), torch.empty(rows, **CUDA)
        guard, dx = guarded_rows(rows, vocab, vocab + pad, dtype)
        space = torch.empty(rr.rr_preference_loss_workspace(rows, pairs), **CUDA, dtype=torch.uint8)
        rr.rr_preference_loss(x, t, offsets, seq_ref, loss, seq, lp, dx, rows, vocab, x.stride(0), dx.stride(0), pairs,
                              hyper, dtype, space, space.numel())
        _, _, _, _, slope, slope_tol = preference(ref, offsets, seq_ref, hyper, rows)
        want, tol = ref.grad(slope, slope_tol, dtype)
        a, b = int(offsets[0]), int(offsets[-1])
        within(dx[a:b], want[a:b], tol[a:b], f"dlogits at {level}")
        guard.check("dlogits")
