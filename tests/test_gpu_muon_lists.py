"""Muon steps over lists longer than a table: the workspace between canaries,
every matrix as in a list of its own."""
import pytest
import torch

from muon_util import COEFS
from step_util import TORCH, Guarded

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


@pytest.mark.parametrize("count,large_first", [(17, False), (160, True), (161, False), (345, True), (345, False)])
def test_long_lists(rr, count, large_first):
    shapes = [(1 + 37 * k % 90, 1 + 53 * k % 130) for k in range(count)]
    shapes[-1 if not large_first else 0] = (700, 300)
    if count > 200:
        shapes[100] = shapes[200] = (0, 4)
    g = torch.Generator(device="cuda").manual_seed(count)

    def normal(dtype):
        return [torch.randn(s, generator=g, **CUDA).to(TORCH[dtype]) for s in shapes]

    params, grads, m, master = normal("bf16"), normal("bf16"), normal("fp32"), normal("fp32")
    start = [[t.clone() for t in ts] for ts in (params, m, master)]
    hyper = rr.rr_muon_hyper(0.1, 0.9, 0.1, 1e-7, 1, 0)
    rows, cols = [s[0] for s in shapes], [s[1] for s in shapes]
    need = rr.rr_orthogonalize_workspace(rows, cols)
    space = Guarded(need, torch.uint8)
    graph = torch.cuda.CUDAGraph()

    def step(p, gr, mo, ma, r, c, w):
        rr.rr_muon(p, gr, mo, ma, r, c, "bf16", "bf16", hyper, COEFS, None, w, w.numel())

    step(params, grads, m, master, rows, cols, space.t)
    torch.cuda.synchronize()
    space.check("workspace")
    got = [[t.clone() for t in ts] for ts in (params, m, master)]
    for k in range(count):
        if rows[k] * cols[k] == 0:
            continue
        p, mo, ma = (ts[k].clone() for ts in start)
        w = torch.empty(rr.rr_orthogonalize_workspace(rows[k:k + 1], cols[k:k + 1]), **CUDA, dtype=torch.uint8)
        step([p], [grads[k]], [mo], [ma], rows[k:k + 1], cols[k:k + 1], w)
        assert torch.equal(p, got[0][k]) and torch.equal(mo, got[1][k]) and torch.equal(ma, got[2][k]), shapes[k]
    # captured and replayed: the tables of one call come one after the other
    for ts, ss in zip((params, m, master), start):
        for t, s in zip(ts, ss):
            t.copy_(s)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(params, grads, m, master, rows, cols, space.t)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for ts, gs in zip((params, m, master), got) for a, b in zip(ts, gs))
    space.check("workspace")
