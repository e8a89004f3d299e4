"""The Muon step's average: its gradient's part is 1 - momentum formed in 64
bits, not from the momentum rounded to binary32."""
import pytest
import torch

from muon_util import COEFS, allowed
from step_util import U24 as u

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


@pytest.mark.parametrize("momentum", [0.0, 0.3, 0.9, 0.95, 0.99, 0.999, 0.9999])
@pytest.mark.parametrize("nesterov", [0, 1])
@pytest.mark.parametrize("shape", [(64, 96), (33, 7)])
def test_average(rr, momentum, nesterov, shape):
    g = torch.Generator(device="cuda").manual_seed(3)
    ws = torch.empty(rr.rr_orthogonalize_workspace([shape[0]], [shape[1]]), **CUDA, dtype=torch.uint8)
    for start in (0.0, 1e-3):
        grad = torch.randn(shape, generator=g, **CUDA)
        m = torch.randn(shape, generator=g, **CUDA) * start
        kept, fresh = momentum * m.double(), (1 - momentum) * grad.double()
        p = torch.zeros(shape, **CUDA)
        rr.rr_muon([p], [grad], [m], None, [shape[0]], [shape[1]], "fp32", "fp32",
                   rr.rr_muon_hyper(1.0, momentum, 0.0, 1e-7, nesterov, rr.RR_MUON_RMS), COEFS, None, ws, ws.numel())
        # factors, products and the sum round once each
        want = kept + fresh
        assert bool(((m.double() - want).abs() <= 2.001 * u * (kept.abs() + fresh.abs()) + u * want.abs()).all())
        # and what is orthogonalised is made of the same factors
        update = fresh + momentum * want if nesterov else want
        o, tol = allowed(update, COEFS)
        step = 0.2 * max(shape) ** 0.5
        # 6u of each value of the update, amplified by at most 3.4445 a step for five steps
        room = step * (10 * tol + 6 * u * 3.4445 ** 5) * float(o.norm()) / o.numel() ** 0.5 + 4 * u * step * o.abs()
        assert bool(((p.double() + step * o).abs() <= room).all())
