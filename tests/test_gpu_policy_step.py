"""A post-training step by the operators together, as a training program calls
them: old log-probabilities, policy or preference loss with its gradient, gradient
norm and clip factor, Muon on the matrices and AdamW on the vectors, against plain
torch in 64 bits."""
import math

import pytest
import torch

from muon_util import COEFS, products

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")
ROWS, WIDTH, INNER, VOCAB, EPS = 96, 64, 160, 1003, 1e-5
LR, ADAM_LR, MAX_NORM = 0.02, 1e-3, 1.0


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


class Net:
    """norm -> two matrices with a residual -> logits, with what its backward needs."""

    def __init__(self, g, dtype):
        def normal(*s):
            return (torch.randn(s, generator=g, **CUDA) * s[-1] ** -0.5).to(dtype)

        self.p = dict(w=torch.ones(WIDTH, **CUDA, dtype=dtype), b=torch.zeros(WIDTH, **CUDA, dtype=dtype),
                      up=normal(INNER, WIDTH), down=normal(WIDTH, INNER), head=normal(VOCAB, WIDTH))

    def clone64(self):
        other = object.__new__(Net)
        other.p = {k: v.double().clone().requires_grad_() for k, v in self.p.items()}
        return other


def forward(rr, p, x):
    h, mean, rstd = torch.empty_like(x), torch.empty(ROWS, **CUDA), torch.empty(ROWS, **CUDA)
    rr.rr_layer_norm(x, p["w"], p["b"], h, mean, rstd, ROWS, WIDTH, WIDTH, WIDTH, EPS, "fp32", "fp32")
    a = h @ p["up"].t()
    y = x + torch.relu(a) @ p["down"].t()
    return y @ p["head"].t(), (h, mean, rstd, a, y)


def backward(rr, p, x, kept, dlogits):
    h, mean, rstd, a, y = kept
    g = {"head": dlogits.t() @ y}
    dy = dlogits @ p["head"]
    r = torch.relu(a)
    g["down"] = dy.t() @ r
    da = (dy @ p["down"]) * (a > 0)
    g["up"] = da.t() @ h
    dh = da @ p["up"]
    g["w"], g["b"], dx = torch.empty_like(p["w"]), torch.empty_like(p["b"]), torch.empty_like(x)
    space = torch.empty(rr.rr_layer_norm_backward_workspace(ROWS, WIDTH), **CUDA, dtype=torch.uint8)
    rr.rr_layer_norm_backward(dh, x, p["w"], mean, rstd, dx, g["w"], g["b"], ROWS, WIDTH, WIDTH, WIDTH, WIDTH, "fp32",
                              "fp32", space, space.numel())
    return {k: v.contiguous() for k, v in g.items()}


def plain_logits(p, x):
    h = torch.nn.functional.layer_norm(x, (WIDTH,), p["w"], p["b"], EPS)
    return (x + torch.relu(h @ p["up"].t()) @ p["down"].t()) @ p["head"].t()


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_step(rr, kind):
    assert not torch.backends.cuda.matmul.allow_tf32
    g = torch.Generator(device="cuda").manual_seed(4)
    net = Net(g, torch.float32)
    want = net.clone64()
    x = torch.randn((ROWS, WIDTH), generator=g, **CUDA)
    target = torch.randint(0, VOCAB, (ROWS,), generator=g, **CUDA)
    target[::7] = -100
    counts = (target >= 0)
    at = torch.where(counts, target, 0)[:, None]
    adv = torch.randn(ROWS, generator=g, **CUDA) + 0.3
    weight = torch.full((ROWS,), 1.0 / ROWS, **CUDA)
    matrices, vectors = ["up", "down", "head"], ["w", "b"]
    rows, cols = [net.p[k].shape[0] for k in matrices], [net.p[k].shape[1] for k in matrices]
    momentum = [torch.zeros_like(net.p[k]) for k in matrices]
    m, v = ([torch.zeros_like(net.p[k]) for k in vectors] for _ in range(2))
    m64 = [t.double() for t in momentum]
    am64, av64 = ([t.double() for t in m] for _ in range(2))
    space = torch.empty(rr.rr_orthogonalize_workspace(rows, cols), **CUDA, dtype=torch.uint8)
    offsets = torch.tensor([0, 20, 48, 75, 96], **CUDA)
    pair_space = torch.empty(rr.rr_preference_loss_workspace(ROWS, 2), **CUDA, dtype=torch.uint8)
    old, ref = torch.empty(ROWS, **CUDA), torch.empty(ROWS, **CUDA)
    logits, _ = forward(rr, net.p, x)
    rr.rr_token_logp(logits, target, old, None, ROWS, VOCAB, VOCAB, 1.0, "fp32")
    ref.copy_(old + 0.1 * torch.randn(ROWS, generator=g, **CUDA))
    first = torch.log_softmax(plain_logits(want.p, x.double()), 1).gather(1, at).view(-1).detach()
    assert float((old - torch.where(counts, first, 0.0)).abs().max()) < 1e-4
    seq_ref = torch.stack([ref[a:b][counts[a:b]].sum() for a, b in zip(offsets.tolist(), offsets.tolist()[1:])])
    loss, token, lp = torch.empty(1, **CUDA), torch.empty(ROWS, **CUDA), torch.empty(ROWS, **CUDA)
    norm, scale = torch.empty(1, **CUDA), torch.empty(1, **CUDA)
    for step in range(1, 4):
        # the operators; the logits are overwritten by their gradient
        logits, kept = forward(rr, net.p, x)
        if kind == "policy":
            hyper = rr.rr_policy_hyper(0.2, 0.28, 0.05, 1.0, 1.0)
            rr.rr_policy_loss(logits, target, old, ref, adv, weight, loss, token, lp, logits, ROWS, VOCAB, VOCAB, VOCAB,
                              hyper, "fp32")
        else:
            hyper = rr.rr_preference_hyper(0.1, 0.05, 0.0, 1.0, 1.0, 0)
            rr.rr_preference_loss(logits, target, offsets, seq_ref, loss, torch.empty(4, **CUDA), lp, logits, ROWS, VOCAB,
                                  VOCAB, VOCAB, 2, hyper, "fp32", pair_space, pair_space.numel())
        grads = backward(rr, net.p, x, kept, logits)
        names = matrices + vectors
        sizes = [net.p[k].numel() for k in names]
        norm_space = torch.empty(rr.rr_grad_norm_workspace(len(sizes)), **CUDA, dtype=torch.uint8)
        rr.rr_grad_norm([grads[k] for k in names], sizes, "fp32", 1.0, MAX_NORM, norm, scale, norm_space, norm_space.numel())
        rr.rr_muon([net.p[k] for k in matrices], [grads[k] for k in matrices], momentum, None, rows, cols, "fp32", "fp32",
                   rr.rr_muon_hyper(LR, 0.95, 0.01, 1e-7, 1, rr.RR_MUON_RMS), COEFS, scale, space, space.numel())
        rr.rr_adamw([net.p[k] for k in vectors], [grads[k] for k in vectors], m, v, None, [WIDTH, WIDTH], "fp32", "fp32",
                    rr.rr_adamw_hyper(ADAM_LR, 0.9, 0.95, 1e-8, 0.01, step), scale)

        # the same in 64 bits
        z = torch.log_softmax(plain_logits(want.p, x.double()), 1).gather(1, at).view(-1)
        if kind == "policy":
            ratio = torch.exp(z - old.double())
            gap = ref.double() - z
            each = -torch.minimum(ratio * adv, ratio.clamp(0.8, 1.28) * adv) + 0.05 * (torch.exp(gap) - gap - 1)
            total = torch.where(counts, each * weight, 0.0).sum()
        else:
            s = torch.stack([torch.where(counts, z, 0.0)[a:b].sum() for a, b in zip(offsets.tolist(), offsets.tolist()[1:])])
            h = 0.1 * ((s[:2] - seq_ref[:2]) - (s[2:] - seq_ref[2:]))
            soft = torch.nn.functional.softplus
            total = (0.95 * soft(-h) + 0.05 * soft(h)).mean()
        d = dict(zip(names, torch.autograd.grad(total, [want.p[k] for k in names])))
        full = torch.sqrt(sum((t * t).sum() for t in d.values()))
        clip = min(1.0, MAX_NORM / (float(full) + 1e-6))
        assert abs(float(loss) - float(total)) <= 1e-4 * max(1.0, abs(float(total)))
        assert abs(float(norm) - float(full)) <= 1e-3 * float(full)
        with torch.no_grad():
            for i, k in enumerate(matrices):
                gk = d[k] * clip
                m64[i] = 0.95 * m64[i] + 0.05 * gk
                o = products(0.05 * gk + 0.95 * m64[i], COEFS)
                p = want.p[k]
                p.mul_(1 - LR * 0.01).sub_(LR * 0.2 * math.sqrt(max(p.shape)) * o)
            for i, k in enumerate(vectors):
                gk = d[k] * clip
                am64[i] = 0.9 * am64[i] + 0.1 * gk
                av64[i] = 0.95 * av64[i] + 0.05 * gk * gk
                upd = am64[i] / (1 - 0.9 ** step) / ((av64[i] / (1 - 0.95 ** step)).sqrt() + 1e-8)
                want.p[k].mul_(1 - ADAM_LR * 0.01).sub_(ADAM_LR * upd)
        # binary32 gradients are off by some 1e-6, which the products amplify by some hundred
        for k in matrices:
            far = float((net.p[k].double() - want.p[k]).norm() / want.p[k].norm())
            assert far < 1e-3, (k, far)
        # where an average is tiny AdamW's first steps are its sign: a vector's values are within a step's size
        for k in vectors:
            assert float((net.p[k].double() - want.p[k]).abs().max()) <= 2.1 * ADAM_LR * step, k
            assert float((net.p[k].double() - want.p[k]).abs().mean()) <= 0.02 * ADAM_LR * step, k
