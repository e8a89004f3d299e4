"""A sharded data-parallel training step on W emulated ranks of one GPU.

    python examples/sharded_step.py --world 4 --steps 30 --states 8

Every rank holds a copy of the weights (bf16) and a microbatch of its own.
One step, with the calls in the order a training program makes them:

  forward     rr_layer_norm before each layer's product, statistics kept
  backward    rr_layer_norm_backward, into the rank's flat gradient buffer
  allreduce   rr_allreduce_twoshot sums the gradients of all ranks
  clip        rr_grad_norm: the norm of the mean gradient and its clip factor
  update      rr_adamw or rr_adamw8 on the rank's shard: its W-th of every
              weight (W divides the width), binary32 master weights and states
              only for that
  allgather   rr_allgather_param_contiguous hands the new weights to all

The model is a small residual network, x <- x + norm(x) V for each layer, fitted
to the outputs of another one with other weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import allgather_rr_allreduce_gb300 as rr  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


class Rank:
    """One rank's buffers.  Weights and gradients are flat, parameter after
    parameter; the shard is the rank's piece of each parameter in turn, as
    rr_allgather_param_contiguous takes it."""

    def __init__(self, r, world, weights, eight):
        shapes = [w.shape for w in weights]
        sizes = [w.numel() for w in weights]
        n = sum(sizes)
        self.param = torch.cat([w.reshape(-1) for w in weights]).to(BF16)
        self.grad, self.summed = torch.zeros(n, device="cuda", dtype=BF16), torch.zeros(n, device="cuda", dtype=BF16)

        def views(flat):
            return [v.view(s) for v, s in zip(flat.split(sizes), shapes)]

        self.params, self.grads = views(self.param), views(self.grad)
        self.pieces = [k // world for k in sizes]
        own = [slice(r * e, (r + 1) * e) for e in self.pieces]
        self.summed_list = list(self.summed.split(sizes))
        self.grad_pieces = [g[o] for g, o in zip(self.summed_list, own)]
        self.shard = torch.cat([p.reshape(-1)[o] for p, o in zip(self.params, own)])
        self.shard_pieces = list(self.shard.split(self.pieces))
        self.masters = [w.reshape(-1)[o].float().clone() for w, o in zip(weights, own)]
        if eight:
            blocks = [-(-e // rr.RR_ADAMW8_BLOCK) for e in self.pieces]
            self.m, self.v = ([torch.zeros(e, device="cuda", dtype=torch.uint8) for e in self.pieces] for _ in range(2))
            self.ms, self.vs = ([torch.zeros(b, device="cuda") for b in blocks] for _ in range(2))
        else:
            self.m, self.v = ([torch.zeros(e, device="cuda") for e in self.pieces] for _ in range(2))
        self.norm, self.scale = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        self.norm_space = torch.empty(rr.rr_grad_norm_workspace(len(sizes)), device="cuda", dtype=torch.uint8)


class Step:
    def __init__(self, world=4, width=256, layers=3, states=8, lr=2e-3, max_norm=1.0, seed=0):
        self.world, self.width, self.layers, self.eight = world, width, layers, states == 8
        self.lr, self.max_norm, self.steps = lr, max_norm, 0
        if width % world:  # every parameter holds width or width^2 elements
            raise ValueError(f"width {width}: {world} ranks do not divide it, and each has an equal piece of every weight")
        g = torch.Generator(device="cuda").manual_seed(seed)

        def network():
            w = []
            for _ in range(layers):
                w += [torch.ones(width, device="cuda"), torch.zeros(width, device="cuda"),
                      torch.randn((width, width), generator=g, device="cuda") * width ** -0.5]
            return w

        self.teacher = [w.to(BF16) for w in network()]
        start = network()
        self.sizes = [w.numel() for w in start]
        self.total = sum(self.sizes)
        self.ranks = [Rank(r, world, start, self.eight) for r in range(world)]
        self.pad = rr.rr_signal_pad_create(world)

    def forward(self, params, x):
        """The network's output and what its backward needs of each layer."""
        rows, kept = x.shape[0], []
        for k in range(self.layers):
            w, b, v = params[3 * k:3 * k + 3]
            h = torch.empty_like(x)
            mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            rr.rr_layer_norm(x, w, b, h, mean, rstd, rows, self.width, self.width, self.width, EPS, "bf16", "bf16")
            kept.append((x, h, mean, rstd))
            x = x + h @ v
        return x, kept

    def backward(self, rank, kept, dx):
        rows = dx.shape[0]
        space = torch.empty(rr.rr_layer_norm_backward_workspace(rows, self.width), device="cuda", dtype=torch.uint8)
        for k in reversed(range(self.layers)):
            x, h, mean, rstd = kept[k]
            w, _, v = rank.params[3 * k:3 * k + 3]
            dw, db, dv = rank.grads[3 * k:3 * k + 3]
            torch.mm(h.t(), dx, out=dv)
            dh = dx @ v.t()
            through = torch.empty_like(dx)
            rr.rr_layer_norm_backward(dh, x, w, mean, rstd, through, dw, db, rows, self.width, self.width, self.width,
                                      self.width, "bf16", "bf16", space, space.numel())
            dx = dx + through

    def run(self, batches):
        """One step on a microbatch for each rank; returns the mean loss."""
        W, losses = self.world, []
        for rank, x in zip(self.ranks, batches):
            want, _ = self.forward(self.teacher, x)
            out, kept = self.forward(rank.params, x)
            diff = (out - want).float()
            losses.append(diff.square().mean())
            self.backward(rank, kept, (diff * (2.0 / diff.numel())).to(BF16))
        rr.rr_allreduce_twoshot(None, [k.grad for k in self.ranks], [k.summed for k in self.ranks], W, self.total,
                                "bf16", 0, self.pad)
        self.steps += 1
        hyper = rr.rr_adamw_hyper(self.lr, 0.9, 0.95, 1e-8, 0.01, self.steps)
        for k in self.ranks:
            rr.rr_grad_norm(k.summed_list, self.sizes, "bf16", 1.0 / W, self.max_norm, k.norm, k.scale, k.norm_space,
                            k.norm_space.numel())
            if self.eight:
                rr.rr_adamw8(k.shard_pieces, k.grad_pieces, k.m, k.ms, k.v, k.vs, k.masters, k.pieces, "bf16", "bf16",
                             hyper, self.steps, k.scale)
            else:
                rr.rr_adamw(k.shard_pieces, k.grad_pieces, k.m, k.v, k.masters, k.pieces, "bf16", "bf16", hyper, k.scale)
        rr.rr_allgather_param_contiguous([k.shard for k in self.ranks], [k.param for k in self.ranks], W,
                                         self.ranks[0].pieces, "bf16", self.pad)
        return torch.stack(losses).mean()

    def close(self):
        self.pad.status()
        self.pad.close()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--world", type=int, default=4)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--states", type=int, choices=(8, 32), default=8)
    a = ap.parse_args()
    step = Step(a.world, states=a.states)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(a.steps):
        batches = [torch.randn((512, step.width), generator=g, device="cuda").to(BF16) for _ in range(a.world)]
        loss = step.run(batches)
        print(f"step {i + 1}: loss {float(loss):.5f}, gradient norm {float(step.ranks[0].norm):.4f}")
    step.close()


if __name__ == "__main__":
    main()
