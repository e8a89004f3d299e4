"""examples/sharded_step.py end to end: the operators and the collectives in one
training step, against the same step in plain binary32 torch."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA GPU")
    from allgather_rr_allreduce_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("sharded_step", os.path.join(ROOT, "examples", "sharded_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def batches(world, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((96, width), generator=g, device="cuda").bfloat16() for _ in range(world)]


def plain_losses(step, steps):
    """The same training in binary32 with torch's autograd, clipping and AdamW."""
    ps = [torch.nn.Parameter(torch.cat([k.masters[i] for k in step.ranks]).view(step.ranks[0].params[i].shape).clone())
          for i in range(len(step.sizes))]
    opt = torch.optim.AdamW(ps, lr=step.lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.01)

    def net(p, x):
        for k in range(step.layers):
            x = x + torch.nn.functional.layer_norm(x, (step.width,), p[3 * k], p[3 * k + 1], 1e-5) @ p[3 * k + 2]
        return x

    out = []
    for i in range(steps):
        loss = torch.stack([(net(ps, x.float()) - net([t.float() for t in step.teacher], x.float())).square().mean()
                            for x in batches(step.world, step.width, i)]).mean()
        opt.zero_grad()
        loss.backward()
        torch.nn.utils.clip_grad_norm_(ps, step.max_norm)
        opt.step()
        out.append(float(loss.detach()))
    return out


@pytest.mark.parametrize("world,states", [(1, 32), (4, 32), (4, 8), (3, 8)])
def test_training_follows_plain_binary32(example, world, states):
    """Activations and gradients round to bf16 (2^-8 relative each), so the loss
    of a step agrees to a few per cent; over 12 steps the two runs see the same
    data and may drift apart by the rounding of the weights and, with 8-bit
    states, of the averages (2^-4 a value, unbiased): 10 %."""
    width = 96
    step = example.Step(world, width=width, layers=2, states=states)
    want = plain_losses(step, 12)
    got = [float(step.run(batches(world, width, i))) for i in range(12)]
    step.close()
    for a, b in zip(got, want):
        assert abs(a - b) <= 0.1 * b, (got, want)
    for k in step.ranks[1:]:
        assert torch.equal(k.param, step.ranks[0].param), "ranks hold different weights"
        assert torch.equal(k.norm, step.ranks[0].norm) and torch.equal(k.scale, step.ranks[0].scale)


def test_a_bad_gradient_costs_no_state(example):
    step = example.Step(2, width=96, layers=1, states=8)
    step.run(batches(2, 96, 0))
    before = [t.clone() for k in step.ranks for t in [k.param, *k.masters, *k.m, *k.v, *k.ms, *k.vs]]
    bad = batches(2, 96, 1)
    bad[1][3, 4] = float("inf")
    step.run(bad)
    after = [t for k in step.ranks for t in [k.param, *k.masters, *k.m, *k.v, *k.ms, *k.vs]]
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    good = float(step.run(batches(2, 96, 2)))
    assert good == good
    step.close()
