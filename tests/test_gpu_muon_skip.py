"""A Muon step whose gradient scale is NaN does no work: nothing but its own
launches happens, and no part of the workspace is written or taken for numbers."""
import pytest
import torch

from muon_util import COEFS

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


@pytest.mark.parametrize("shapes", [[(40, 70)], [(300, 280), (1000, 130)], [(30 + k, 64) for k in range(170)]])
@pytest.mark.parametrize("masters", [False, True])
def test_skipped_step(rr, shapes, masters):
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(dtype=torch.float32):
        return [torch.randn(s, generator=g, **CUDA).to(dtype) for s in shapes]

    params, grads, m, master = normal(torch.bfloat16), normal(torch.bfloat16), normal(), normal() if masters else None
    before = [t.clone() for t in params + m + (master or [])]
    rows, cols = [s[0] for s in shapes], [s[1] for s in shapes]
    ws = torch.full((rr.rr_orthogonalize_workspace(rows, cols),), 0xA5, **CUDA, dtype=torch.uint8)
    scale = torch.full((1,), float("nan"), **CUDA)

    def step():
        rr.rr_muon(params, grads, m, master, rows, cols, "bf16", "bf16", rr.rr_muon_hyper(0.1, 0.9, 0.1, 1e-7, 1, 0), COEFS,
                   scale, ws, ws.numel())

    step()
    assert all(torch.equal(a, b) for a, b in zip(before, params + m + (master or [])))
    assert bool((ws == 0xA5).all())
    scale.fill_(0.5)  # the next step is an ordinary one
    step()
    assert not any(torch.equal(a, b) for a, b in zip(before, params + m + (master or [])))
    assert all(bool(torch.isfinite(t.float()).all()) for t in params + m + (master or []))
