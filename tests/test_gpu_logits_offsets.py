"""Offsets of a preference loss anywhere in 64 bits are kept to the rows: no row
before the first or behind the last is read or written, and sequences whose own
offsets are in order keep their values."""
import pytest
import torch

from logits_util import Reference, make
from step_util import Guarded

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")
MOST, LEAST = 2 ** 63 - 1, -2 ** 63


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


@pytest.mark.parametrize("rows,vocab", [(6, 50), (700, 9), (3, 40000)])
@pytest.mark.parametrize("offsets,read", [
    ((MOST, MOST, MOST), (0, 0)), ((LEAST, LEAST, LEAST), (0, 0)), ((MOST - 3, 2, LEAST), (0, 0)), ((0, 2, LEAST), (0, 0)),
    ((MOST, 2, 3), (0, 0)), ((LEAST, 2, MOST), (0, 2)), ((LEAST, MOST, MOST), (0, 3)), ((0, MOST - 100, MOST), (0, 3)),
    ((-1, 2, 1 << 62), (0, 2)),
])
def test_offsets_anywhere(rr, rows, vocab, offsets, read):
    x, t, _ = make(rows, vocab, "fp32", seed=1, ignored=0)
    o = torch.tensor(offsets, **CUDA)
    loss, seq = torch.empty(1, **CUDA), torch.empty(2, **CUDA)
    lp, dx = Guarded(rows, torch.float32), Guarded(rows * vocab, torch.float32)
    need = rr.rr_preference_loss_workspace(rows, 1)
    space = Guarded(need, torch.uint8)
    for grad in (None, dx.t):
        rr.rr_preference_loss(x, t, o, None, loss, seq, lp.t, grad, rows, vocab, vocab, vocab, 1,
                              rr.rr_preference_hyper(0.1, 0.0, 0.0, 1.0, 1.0, 0), "fp32", space.t, need)
        torch.cuda.synchronize()
        for g in (lp, dx, space):
            g.check()
    if read[1] == 0:  # no sequence in order: unspecified, but in bounds
        return
    a, b = read[0], rows if read[1] == 3 else read[1]
    ref = Reference(x, t, 1.0)
    tol = float(ref.logp_tol[a:b].sum() + 2.0 ** -24 * ref.logp[a:b].abs().sum())
    assert abs(float(seq[0]) - float(ref.logp[a:b].sum())) <= tol
