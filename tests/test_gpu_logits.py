"""Log-probabilities of tokens and the losses over logits against their formulas in 64 bits."""
import math

import pytest
import torch

from logits_util import Reference, make, policy
from step_util import BYTES, TORCH, U24 as u, Guarded, within

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


def logp(rr, x, t, inv_t=1.0, dtype="bf16"):
    rows, vocab = x.shape
    out, lse = torch.full((2, rows), 7.0, **CUDA)
    rr.rr_token_logp(x, t, out, lse, rows, vocab, x.stride(0), inv_t, dtype)
    return out, lse


def guarded_rows(rows, vocab, stride, dtype, shift=0):
    g = Guarded((rows - 1) * stride + vocab, TORCH[dtype], shift)
    return g, g.t.as_strided((rows, vocab), (stride, 1))


def gaps_untouched(g, rows, vocab, stride):
    """What lies between rows of a wider buffer keeps its canary."""
    raw = g.t.view(torch.uint8)
    eb = g.t.element_size()
    for r in range(rows - 1):
        gap = raw[(r * stride + vocab) * eb:(r + 1) * stride * eb]
        assert bool((gap == 0xA5).all())


SHAPES = [(1, 1), (3, 2), (5, 7), (300, 8), (2, 31), (33, 100), (700, 257), (9, 1000), (1, 4097), (40, 4096), (170, 8192),
          (3, 50021), (500, 20011), (1, 131072), (8, 131072), (60, 65536), (200, 32000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_logp_and_gradient(rr, rows, vocab, dtype):
    for pad, shift, inv_t in ((0, 0, 1.0), (3, 1, 0.75)):
        x, t, g = make(rows, vocab, dtype, seed=rows * 31 + vocab, pad=pad, shift=shift)
        ref = Reference(x, t, inv_t)
        got, lse = logp(rr, x, t, inv_t, dtype)
        within(got, ref.logp, torch.where(ref.counts, ref.logp_tol, 0.0), "logp")
        within(lse, ref.lse, torch.where(ref.counts, ref.lse_tol, 0.0), "lse")
        again, _ = logp(rr, x, t, inv_t, dtype)
        assert torch.equal(got, again)
        d = torch.randn(rows, generator=g, **CUDA)
        for dpad, dshift in ((pad, shift), (pad + 2, shift + 1)):
            guard, dx = guarded_rows(rows, vocab, vocab + dpad, dtype, dshift)
            rr.rr_token_logp_backward(x, t, lse, d, dx, rows, vocab, x.stride(0), dx.stride(0), inv_t, dtype)
            # the base lse / inv_t and the difference from it round at the size of the logits
            extra = u * 6 * (ref.lse.abs() + ref.z.abs().amax(1)) + ref.lse_tol
            want, tol = ref.grad(d.double(), torch.zeros_like(ref.lse), dtype, extra)
            within(dx, want, tol, "dlogits")
            guard.check("dlogits")
            gaps_untouched(guard, rows, vocab, vocab + dpad)


def policy_inputs(ref, g, kl=True):
    n = ref.logp.numel()
    d = torch.randn(n, generator=g, **CUDA) * 0.2
    for border in (math.log(0.8), math.log(1.28)):
        d = torch.where((d - border).abs() < 1e-3, d + 4e-3, d)
    old = (ref.logp - d).float()
    kl_ref = (ref.logp - torch.randn(n, generator=g, **CUDA) * 0.3).float() if kl else None
    adv = torch.randn(n, generator=g, **CUDA) + 0.3
    weight = torch.rand(n, generator=g, **CUDA) / n
    return old, kl_ref, adv, weight


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_policy_loss(rr, rows, vocab, dtype):
    for k, (pad, dpad, inv_t) in enumerate(((0, 0, 1.0), (3, 0, 1.25), (0, 5, 0.5))):
        x, t, g = make(rows, vocab, dtype, seed=rows + vocab, pad=pad)
        ref = Reference(x, t, inv_t)
        old, kl_ref, adv, weight = policy_inputs(ref, g, kl=k != 1)
        if k == 2:
            old = weight = None
        hyper = rr.rr_policy_hyper(0.2, 0.28, 0.05, inv_t, 64.0)
        token, lp = torch.full((2, rows), 7.0, **CUDA)
        loss = torch.zeros(1, **CUDA)
        guard, dx = guarded_rows(rows, vocab, vocab + dpad, dtype)
        rr.rr_policy_loss(x, t, old, kl_ref, adv, weight, loss, token, lp, dx, rows, vocab, x.stride(0), dx.stride(0),
                          hyper, dtype)
        want, tol, slope, slope_tol = policy(ref, old, kl_ref, adv, weight, hyper)
        within(lp, ref.logp, torch.where(ref.counts, ref.logp_tol, 0.0), "logp")
        within(token, want, tol, "token_loss")
        within(loss, want.sum().view(1), (tol.sum() + 2 * u * want.sum().abs()).view(1), "loss")
        grad, gtol = ref.grad(slope * 64, slope_tol * 64, dtype)
        within(dx, grad, gtol, "dlogits")
        guard.check("dlogits")
        gaps_untouched(guard, rows, vocab, vocab + dpad)
        # without the gradient, and without the sum
        token2, lp2 = torch.full((2, rows), 7.0, **CUDA)
        rr.rr_policy_loss(x, t, old, kl_ref, adv, weight, None, token2, lp2, None, rows, vocab, x.stride(0), 0, hyper, dtype)
        assert torch.equal(token, token2) and torch.equal(lp, lp2)
        # in place
        y = x.clone(memory_format=torch.contiguous_format)
        rr.rr_policy_loss(y, t, old, kl_ref, adv, weight, loss, token2, lp2, y, rows, vocab, vocab, vocab, hyper, dtype)
        within(y, grad, gtol, "dlogits in place")


def test_policy_gradient_by_differences(rr):
    rows, vocab = 24, 97
    x, t, g = make(rows, vocab, "fp32", seed=5, ignored=0.1)
    ref = Reference(x, t, 0.8)
    old, kl_ref, adv, weight = policy_inputs(ref, g)
    hyper = rr.rr_policy_hyper(0.2, 0.28, 0.3, 0.8, 1.0)
    token, lp = torch.empty((2, rows), **CUDA)
    dx = torch.empty_like(x)
    rr.rr_policy_loss(x, t, old, kl_ref, adv, weight, None, token, lp, dx, rows, vocab, vocab, vocab, hyper, "fp32")
    for _ in range(8):
        v = torch.randn(x.shape, generator=g, **CUDA).double()
        h = 1e-5  # no ratio within 1e-3 of a border: both sides stay on their branch

        def at(s):
            return policy(Reference(x.double() + s * h * v, t, 0.8), old, kl_ref, adv, weight, hyper)[0].sum()

        slope = float(at(1) - at(-1)) / (2 * h)
        along = float((dx.double() * v).sum())
        scale = float((dx.double().abs() * v.abs()).sum())
        # the difference's own error: h^2 times third derivatives of order one a row, and 1e-16 / h
        assert abs(slope - along) <= 1e-5 * scale + 1e-8, (slope, along)


def pair_case(rows_of, vocab, dtype, seed, lead=2, tail=3, pad=0, shift=0):
    offsets = [lead]
    for n in rows_of:
        offsets.append(offsets[-1] + n)
    x, t, g = make(offsets[-1] + tail, vocab, dtype, seed, pad=pad, shift=shift)
    return x, t, torch.tensor(offsets, **CUDA), g


def preference(ref, offsets, seq_ref, hyper, rows):
    """loss, seq_logp, each row's slope, and tolerances."""
    o = offsets.tolist()
    pairs = (len(o) - 1) // 2
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    s, st, counts = [], [], []
    for a, b in zip(o, o[1:]):
        n = max(1, int(ref.counts[a:b].sum())) if hyper.average else 1
        s.append(ref.logp[a:b].sum() / n)
        st.append(torch.where(ref.counts[a:b], ref.logp_tol[a:b], 0.0).sum() / n + u * s[-1].abs())
        counts.append(n)
    s, st = torch.stack(s), torch.stack(st)
    r = torch.zeros_like(s) if seq_ref is None else seq_ref.double()
    beta, eps, margin = f32(hyper.beta), f32(hyper.label_smoothing), f32(hyper.margin)
    h = beta * ((s[:pairs] - r[:pairs]) - (s[pairs:] - r[pairs:])) - margin
    h_tol = beta * (st[:pairs] + st[pairs:]) + u * h.abs()
    soft = torch.nn.functional.softplus
    sp = lambda v: torch.where(v > 30, v + torch.exp(-v), soft(v, threshold=1e9))  # noqa: E731
    each = (1 - eps) * sp(-h) + eps * sp(h)
    each_tol = h_tol + 12 * u * (sp(-h) + sp(h))
    dh = (eps * torch.sigmoid(h) - (1 - eps) * torch.sigmoid(-h)) * beta / pairs * hyper.grad_scale
    dh_tol = (h_tol * 0.25 + 16 * u) * beta / pairs * hyper.grad_scale
    slope, slope_tol = torch.zeros(rows, **CUDA).double(), torch.zeros(rows, **CUDA).double()
    for k in range(2 * pairs):
        sign = 1 if k < pairs else -1
        slope[o[k]:o[k + 1]] = sign * dh[k % pairs] / counts[k]
        slope_tol[o[k]:o[k + 1]] = dh_tol[k % pairs] / counts[k]
    return each.mean().view(1), (each_tol.mean() + u * each.mean()).view(1), s, st, slope, slope_tol


PAIRS = [((1, 1), 5), ((4, 0), 100), ((0, 0), 33), ((20, 30), 32000), ((17, 3, 0, 9, 1, 40), 1025),
         ((60, 41, 12, 55, 7, 70, 33, 20), 50021), ((900, 700, 800, 1), 512), ((40, 60), 131072)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lens,vocab", PAIRS)
def test_preference_loss(rr, lens, vocab, dtype):
    for k, (pad, shift, average, inv_t) in enumerate(((0, 0, 0, 1.0), (3, 1, 1, 0.75))):
        x, t, offsets, g = pair_case(lens, vocab, dtype, seed=vocab + k, pad=pad, shift=shift)
        rows, pairs = x.shape[0], len(lens) // 2
        ref = Reference(x, t, inv_t)
        sums = torch.stack([ref.logp[a:b].sum() for a, b in zip(offsets.tolist(), offsets.tolist()[1:])])
        seq_ref = None if k else (sums + torch.randn(len(lens), generator=g, **CUDA) * 8).float()
        hyper = rr.rr_preference_hyper(2.0 if average else 0.1, 0.1, 0.5 if average else 0.0, inv_t, 256.0, average)
        loss, seq = torch.empty(1, **CUDA), torch.empty(2 * pairs, **CUDA)
        lp = torch.full((rows,), 7.0, **CUDA)
        guard, dx = guarded_rows(rows, vocab, vocab + 2 * pad, dtype)
        guard.t.fill_(3.0)
        space = torch.empty(rr.rr_preference_loss_workspace(rows, pairs), **CUDA, dtype=torch.uint8)
        args = (t, offsets, seq_ref, loss, seq, lp)
        rr.rr_preference_loss(x, *args, dx, rows, vocab, x.stride(0), dx.stride(0), pairs, hyper, dtype, space,
                              space.numel())
        want, tol, s, st, slope, slope_tol = preference(ref, offsets, seq_ref, hyper, rows)
        a, b = int(offsets[0]), int(offsets[-1])
        within(lp[a:b], ref.logp[a:b], torch.where(ref.counts, ref.logp_tol, 0.0)[a:b], "logp")
        within(seq, s, st, "seq_logp")
        within(loss, want, tol, "loss")
        extra = u * 6 * (ref.lse.abs() + ref.z.abs().amax(1)) + ref.lse_tol
        grad, gtol = ref.grad(slope, slope_tol, dtype, extra)
        within(dx[a:b], grad[a:b], gtol[a:b], "dlogits")
        # rows of no sequence are left as they were
        for edge in (slice(0, a), slice(b, rows)):
            assert bool((lp[edge] == 7).all()) and bool((dx[edge] == 3).all())
        guard.check("dlogits")
        # loss alone
        loss2, seq2, lp2 = torch.empty(1, **CUDA), torch.empty(2 * pairs, **CUDA), torch.full((rows,), 7.0, **CUDA)
        rr.rr_preference_loss(x, t, offsets, seq_ref, loss2, seq2, lp2, None, rows, vocab, x.stride(0), 0, pairs, hyper,
                              dtype, space, space.numel())
        assert torch.equal(loss, loss2) and torch.equal(seq, seq2) and torch.equal(lp, lp2)
        # in place
        y = x.clone(memory_format=torch.contiguous_format)
        rr.rr_preference_loss(y, *args, y, rows, vocab, vocab, vocab, pairs, hyper, dtype, space, space.numel())
        within(y[a:b], grad[a:b], gtol[a:b], "dlogits in place")
        assert torch.equal(y[:a], x[:a]) and torch.equal(y[b:], x[b:])


def test_preference_gradient_by_differences(rr):
    x, t, offsets, g = pair_case((6, 4, 3, 9), 61, "fp32", seed=3)
    rows, pairs = x.shape[0], 2
    hyper = rr.rr_preference_hyper(0.5, 0.1, 0.2, 1.0, 1.0, 0)
    seq_ref = -torch.rand(4, generator=g, **CUDA) * 20
    out = [torch.empty(1, **CUDA), torch.empty(4, **CUDA), torch.empty(rows, **CUDA)]
    dx = torch.zeros_like(x)
    space = torch.empty(rr.rr_preference_loss_workspace(rows, pairs), **CUDA, dtype=torch.uint8)
    rr.rr_preference_loss(x, t, offsets, seq_ref, *out, dx, rows, 61, 61, 61, pairs, hyper, "fp32", space, space.numel())
    for _ in range(8):
        v = torch.randn(x.shape, generator=g, **CUDA).double()
        h = 1e-5

        def at(s):
            return preference(Reference(x.double() + s * h * v, t, 1.0), offsets, seq_ref, hyper, rows)[0]

        slope = float(at(1) - at(-1)) / (2 * h)
        along = float((dx.double() * v).sum())
        scale = float((dx.double().abs() * v.abs()).sum())
        assert abs(slope - along) <= 1e-5 * scale + 1e-8, (slope, along)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [5, 1000, 40000])
def test_masked_and_special_values(rr, dtype, vocab):
    """-inf masks, the type's lowest value, infinities and NaN, rows of nothing but -inf."""
    rows = 8
    x, t, g = make(rows, vocab, dtype, seed=vocab, ignored=0)
    inf, low = float("inf"), torch.finfo(TORCH[dtype]).min
    keep = torch.zeros(rows, vocab, dtype=torch.bool, **CUDA).scatter_(1, t[:, None], True)
    half = torch.rand((rows, vocab), generator=g, **CUDA) < 0.5
    x[0].masked_fill_(half[0] & ~keep[0], -inf)
    x[1].masked_fill_(~keep[1], -inf)            # only the target is left
    x[2].fill_(-inf)                             # nothing is left
    x[3].masked_fill_(half[3] & ~keep[3], low)
    x[4].masked_fill_(keep[4], -inf)             # the target is masked
    x[5, vocab // 2] = inf
    x[6, vocab - 1] = float("nan")
    x[7].fill_(low)
    got, lse = logp(rr, x, t, 1.0, dtype)
    ref = Reference(x, t, 1.0)
    tol = torch.where(torch.isfinite(ref.logp_tol), ref.logp_tol, 1.0)
    want = torch.where(torch.isnan(ref.logp), float("nan"), ref.logp)
    within(got, want, tol, "logp")
    assert torch.isnan(got[[2, 5, 6]]).all() and got[4] == -inf and got[1] == 0
    adv = torch.ones(rows, **CUDA)
    token, lp, dx = torch.empty(rows, **CUDA), torch.empty(rows, **CUDA), torch.empty_like(x)
    hyper = rr.rr_policy_hyper(0.2, 0.2, 0.0, 1.0, 1.0)
    old = torch.full((rows,), -3.0, **CUDA)
    rr.rr_policy_loss(x, t, old, None, adv, None, None, token, lp, dx, rows, vocab, vocab, vocab, hyper, dtype)
    assert torch.isnan(dx[[2, 5, 6]]).all() and torch.isnan(token[[2, 5, 6]]).all()
    fine = [0, 1, 3, 4, 7]
    assert torch.isfinite(dx[fine].float()).all() and token[4] == 0 and bool((dx[4] == 0).all())
    _, _, slope, slope_tol = policy(ref, old, None, adv, None, hyper)
    want, gtol = ref.grad(slope, slope_tol, dtype)
    rows_ = [0, 1, 3, 7]
    gap_free = torch.where(torch.isfinite(gtol), gtol, 0.0)  # a masked place has gap inf, probability 0: exactly 0
    within(dx[rows_], want[rows_], gap_free[rows_], "dlogits")
    masked = torch.isinf(x[0])
    assert bool((dx[0][masked] == 0).all())


def test_offsets_past_32_bits(rr):
    """Rows beyond 2^31 and 2^32 elements."""
    rows, vocab = 33000, 131072  # 4.3e9 elements of bf16
    x = torch.zeros((rows, vocab), **CUDA, dtype=torch.bfloat16)
    pick = [0, 16383, 16384, 32767, 32768, rows - 1]
    g = torch.Generator(device="cuda").manual_seed(1)
    x[pick] = (torch.randn((len(pick), vocab), generator=g, **CUDA) * 2).bfloat16()
    t = torch.randint(0, vocab, (rows,), generator=g, **CUDA)
    adv = torch.ones(rows, **CUDA)
    token, lp = torch.empty((2, rows), **CUDA)
    hyper = rr.rr_policy_hyper(0.2, 0.2, 0.0, 1.0, 1.0)
    ref = Reference(x[pick], t[pick], 1.0)
    rr.rr_policy_loss(x, t, None, None, adv, None, None, token, lp, x, rows, vocab, vocab, vocab, hyper, "bf16")
    within(lp[pick], ref.logp, ref.logp_tol, "logp")
    want, tol = ref.grad(-torch.ones(len(pick), **CUDA).double(), torch.zeros(len(pick), **CUDA).double(), "bf16")
    within(x[pick], want, tol, "dlogits")
    other = torch.ones(rows, dtype=torch.bool, **CUDA)
    other[pick] = False
    within(lp[other], torch.full((int(other.sum()),), -math.log(vocab), **CUDA).double(),
           torch.full((1,), 300 * u, **CUDA).double(), "rows of zeros")


def test_streams_and_graphs(rr):
    rows, vocab = 37, 33000
    x, t, g = make(rows, vocab, "bf16", seed=9)
    ref = Reference(x, t, 1.0)
    old, kl_ref, adv, weight = policy_inputs(ref, g)
    hyper = rr.rr_policy_hyper(0.2, 0.28, 0.05, 1.0, 1.0)

    def buffers():
        return torch.empty(1, **CUDA), torch.empty(rows, **CUDA), torch.empty(rows, **CUDA), torch.empty_like(x)

    def call(x, out):
        rr.rr_policy_loss(x, t, old, kl_ref, adv, weight, *out, rows, vocab, vocab, vocab, hyper, "bf16")

    want = buffers()
    call(x, want)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [buffers() for _ in side]
    torch.cuda.synchronize()
    for s, o in zip(side, outs):  # two calls at once
        with torch.cuda.stream(s):
            for _ in range(5):
                call(x, o)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    graph, o, y = torch.cuda.CUDAGraph(), buffers(), torch.zeros_like(x)
    with torch.cuda.graph(graph):
        call(y, o)
    y.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, want))

    offsets = torch.tensor([0, 9, 20, 30, 37], **CUDA)
    hyper2 = rr.rr_preference_hyper(0.1, 0.0, 0.0, 1.0, 1.0, 0)
    space = [torch.empty(rr.rr_preference_loss_workspace(rows, 2), **CUDA, dtype=torch.uint8) for _ in range(2)]

    def pair(x, out, k):
        rr.rr_preference_loss(x, t, offsets, None, out[0], out[1], out[2], out[3], rows, vocab, vocab, vocab, 2, hyper2,
                              "bf16", space[k], space[k].numel())

    def pair_buffers():
        return torch.empty(1, **CUDA), torch.empty(4, **CUDA), torch.empty(rows, **CUDA), torch.empty_like(x)

    want = pair_buffers()
    pair(x, want, 0)
    torch.cuda.synchronize()
    graph, o = torch.cuda.CUDAGraph(), pair_buffers()
    with torch.cuda.graph(graph):
        pair(y, o, 1)
    y.zero_()
    graph.replay()
    y.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_empty_calls(rr):
    hyper = rr.rr_policy_hyper(0.2, 0.2, 0.0, 1.0, 1.0)
    loss = torch.full((1,), 5.0, **CUDA)
    rr.rr_token_logp(None, None, None, None, 0, 10, 10, 1.0, "bf16")
    rr.rr_token_logp_backward(None, None, None, None, None, 0, 10, 10, 10, 1.0, "bf16")
    rr.rr_policy_loss(None, None, None, None, None, None, loss, None, None, None, 0, 10, 10, 10, hyper, "bf16")
    assert float(loss) == 0
    seq, offsets = torch.full((2,), 5.0, **CUDA), torch.zeros(3, **CUDA, dtype=torch.int64)
    space = torch.empty(rr.rr_preference_loss_workspace(0, 1), **CUDA, dtype=torch.uint8)
    rr.rr_preference_loss(None, None, offsets, None, loss, seq, None, None, 0, 10, 10, 10, 1,
                          rr.rr_preference_hyper(0.1, 0.0, 0.0, 1.0, 1.0, 0), "bf16", space, space.numel())
    assert bool((seq == 0).all()) and abs(float(loss) - math.log(2)) < 1e-6


def test_offsets_out_of_range_stay_in_bounds(rr):
    """Offsets outside the rows are kept to them: nothing outside the buffers is touched."""
    x, t, _ = make(6, 50, "fp32", seed=1)
    offsets = torch.tensor([-5, 2, 1 << 40], **CUDA)
    loss, seq, lp = torch.empty(1, **CUDA), torch.empty(2, **CUDA), Guarded(6, torch.float32)
    guard, dx = guarded_rows(6, 50, 50, "fp32")
    need = rr.rr_preference_loss_workspace(6, 1)
    space = Guarded(need, torch.uint8)
    rr.rr_preference_loss(x, t, offsets, None, loss, seq, lp.t, dx, 6, 50, 50, 50, 1,
                          rr.rr_preference_hyper(0.1, 0.0, 0.0, 1.0, 1.0, 0), "fp32", space.t, need)
    torch.cuda.synchronize()
    for gd in (lp, guard, space):
        gd.check()
    assert torch.isfinite(loss).all()


def test_element_sizes_match():
    assert BYTES == {k: torch.empty((), dtype=v).element_size() for k, v in TORCH.items()}
