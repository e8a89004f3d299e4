"""Newton-Schulz products and the Muon step against the formulas in 64 bits."""
import math

import pytest
import torch

from muon_util import COEFS, allowed, near, products
from step_util import TORCH, U, U24, Guarded

pytestmark = pytest.mark.gpu
CUDA = dict(device="cuda")


@pytest.fixture(scope="module")
def rr():
    import allgather_rr_allreduce_gb300 as m
    return m


def space(rr, rows, cols):
    return torch.empty(max(1, rr.rr_orthogonalize_workspace(rows, cols)), **CUDA, dtype=torch.uint8)


def orthogonalize(rr, xs, ydt="fp32", coefs=COEFS, eps=1e-7, ys=None):
    names = {v: k for k, v in TORCH.items()}
    rows, cols = [x.shape[0] for x in xs], [x.shape[1] for x in xs]
    ys = [torch.empty(x.shape, **CUDA, dtype=TORCH[ydt]) for x in xs] if ys is None else ys
    w = space(rr, rows, cols)
    w.fill_(0xFF)  # a workspace of NaN
    rr.rr_orthogonalize(xs, ys, rows, cols, names[xs[0].dtype], ydt, coefs, eps, w, w.numel())
    return ys


def matrix(shape, seed, kind="noise", dtype="fp32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, n = shape
    x = torch.randn(shape, generator=g, **CUDA)
    if kind == "low rank":  # a few directions carry most of it
        k = min(8, m, n)
        x = x + torch.randn((m, k), generator=g, **CUDA) @ torch.randn((k, n), generator=g, **CUDA)
    if kind == "positive":
        x = x.abs() + 0.1
    return x.to(TORCH[dtype])


SHAPES = [(1, 1), (1, 300), (300, 1), (2, 3), (63, 65), (64, 64), (65, 63), (128, 128), (129, 127), (100, 1000), (1000, 100),
          (255, 257), (256, 256), (257, 511), (513, 2050), (1000, 777), (384, 4100), (1300, 1290)]


@pytest.mark.parametrize("kind", ["noise", "low rank", "positive"])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(rr, shape, kind):
    x = matrix(shape, seed=shape[0] * 7 + shape[1], kind=kind)
    want, tol = allowed(x, COEFS)
    y, = orthogonalize(rr, [x])
    near(y, want, tol, U["fp32"], kind)
    again, = orthogonalize(rr, [x])
    assert torch.equal(y, again)
    flipped, = orthogonalize(rr, [x.t().contiguous()])
    # The same products on the short side, but not bit for bit: squares are added in the
    # order of memory, eight at a time in binary32, so the norms may differ by 4u.
    near(flipped.t(), want, tol, U["fp32"], "transposed")


@pytest.mark.parametrize("xdt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ydt", ["bf16", "fp16", "fp32"])
def test_types_and_alignment(rr, xdt, ydt):
    """A list of matrices that start at any element, results between canaries."""
    shapes = [(70, 130), (130, 70), (33, 64), (256, 512), (7, 9)]
    xs, guards = [], []
    for k, s in enumerate(shapes):
        flat = torch.empty(s[0] * s[1] + k, **CUDA, dtype=TORCH[xdt])
        x = flat[k:].view(s)
        x.copy_(matrix(s, seed=k))
        xs.append(x)
        guards.append(Guarded(s[0] * s[1], TORCH[ydt], (2 * k + 1) % 5))
    ys = [g.t.view(s) for g, s in zip(guards, shapes)]
    orthogonalize(rr, xs, ydt, ys=ys)
    for x, y, g in zip(xs, ys, guards):
        want, tol = allowed(x, COEFS)
        near(y, want, tol, U[ydt], f"{tuple(x.shape)}")
        g.check()


@pytest.mark.parametrize("coefs", [[(1.5, -0.5, 0.0)], [(2.0, -1.5, 0.5)] * 12, [(3.4445, -4.7750, 2.0315)] * 2 + [(1.875, -1.25, 0.375)] * 4,
                                   [(0.0, 1.0, 0.0)], [(0.5, 0.25, -1.0)]])
def test_coefficients(rr, coefs):
    x = matrix((200, 333), seed=3)
    want, tol = allowed(x, coefs)
    y, = orthogonalize(rr, [x], coefs=coefs)
    near(y, want, tol, U["fp32"])


def test_singular_values(rr):
    for x in (matrix((300, 500), 1), matrix((500, 300), 2, "low rank")):
        y, = orthogonalize(rr, [x])
        s = torch.linalg.svdvals(y.double())
        start = torch.linalg.svdvals(x.double())
        moved = start / start.norm() > 1e-2
        assert float(s[moved].min()) > 0.65 and float(s.max()) < 1.25
        # twelve steps of a cubic that converges to 1
        y, = orthogonalize(rr, [x], coefs=[(3.4445, -4.7750, 2.0315)] * 5 + [(1.5, -0.5, 0.0)] * 8)
        s = torch.linalg.svdvals(y.double())
        assert float((s - 1).abs().max()) < 1e-4


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-12, 1.0, 1e12, 1e30, 1e37])
def test_sizes_of_values(rr, scale):
    """The norm's squares leave binary32's range at both ends."""
    x = (matrix((90, 130), seed=4).double() * scale).float()
    want, tol = allowed(x, COEFS, eps=0.0)
    y, = orthogonalize(rr, [x], eps=0.0)
    near(y, want, tol, U["fp32"])


def test_zeros_and_values_that_are_not_finite(rr):
    x = matrix((70, 90), seed=1)
    zero = torch.zeros_like(x)
    y, = orthogonalize(rr, [zero])
    assert bool((y == 0).all())
    one = zero.clone()
    one[3, 4] = -2.0
    want, tol = allowed(one, COEFS)
    y, = orthogonalize(rr, [one])
    near(y, want, tol, U["fp32"])
    bad, inf = x.clone(), x.clone()
    bad[5, 6] = float("nan")
    inf[5, 6] = float("inf")
    ys = orthogonalize(rr, [bad, x, inf])
    assert bool(torch.isnan(ys[0]).all()) and bool(torch.isnan(ys[2]).all())
    want, tol = allowed(x, COEFS)
    near(ys[1], want, tol, U["fp32"], "beside them")


def test_lists(rr):
    """Longer than one launch's table, with empty matrices in it."""
    shapes = [(1 + 37 * k % 90, 1 + 53 * k % 130) for k in range(331)]
    shapes[5] = shapes[200] = (0, 4)
    shapes[330] = (7, 0)
    xs = [matrix(s, seed=k) if s[0] * s[1] else torch.empty(s, **CUDA) for k, s in enumerate(shapes)]
    ys = orthogonalize(rr, xs)
    for k in [0, 1, 15, 16, 17, 159, 160, 161, 162, 163, 319, 320, 321, 322, 329]:
        if shapes[k][0] * shapes[k][1]:
            alone, = orthogonalize(rr, [xs[k]])
            assert torch.equal(alone, ys[k]), shapes[k]
            want, tol = allowed(xs[k], COEFS)
            near(ys[k], want, tol, U["fp32"], str(shapes[k]))


def test_in_place_and_nothing_to_do(rr):
    x = matrix((130, 100), seed=8)
    want, = orthogonalize(rr, [x])
    orthogonalize(rr, [x], ys=[x])
    assert torch.equal(x, want)
    rr.rr_orthogonalize([], [], [], [], "fp32", "fp32", COEFS, 1e-7, None, 0)
    rr.rr_orthogonalize([None], [None], [0], [5], "fp32", "fp32", COEFS, 1e-7, None, 0)


def muon_want(p, g, m, master, shape, hyper, scale, coefs=COEFS):
    """New weights and momentum in 64 bits, and the weights' tolerance."""
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    mu = f32(hyper.momentum)
    g = g.double() * (1.0 if scale is None else float(scale))
    m = mu * m.double() + (1 - mu) * g
    u = (1 - mu) * g + mu * m if hyper.nesterov else m
    o, tol = allowed(u, coefs, hyper.eps)
    r, c = shape
    step = hyper.lr * (0.2 * math.sqrt(max(r, c)) if hyper.adjust else math.sqrt(max(1.0, r / c)))
    w = (p if master is None else master).double()
    return (1 - hyper.lr * hyper.weight_decay) * w - step * o, m, step * tol * float(o.norm())


@pytest.mark.parametrize("pdt,gdt,masters", [("fp32", "fp32", False), ("bf16", "bf16", True), ("bf16", "fp32", False),
                                             ("fp16", "fp16", True), ("fp16", "bf16", False)])
@pytest.mark.parametrize("nesterov,adjust", [(1, 0), (0, 1)])
def test_muon(rr, pdt, gdt, masters, nesterov, adjust):
    shapes = [(96, 200), (200, 96), (65, 33), (300, 300), (1, 50)]
    g = torch.Generator(device="cuda").manual_seed(11)
    w = [torch.randn(s, generator=g, **CUDA) * 0.05 for s in shapes]
    params = [v.to(TORCH[pdt]) for v in w]
    master = w if masters else None
    m = [torch.randn(s, generator=g, **CUDA) * 1e-3 for s in shapes]
    scale = torch.full((1,), 0.37, **CUDA)
    hyper = rr.rr_muon_hyper(0.02, 0.95, 0.1, 1e-7, nesterov, adjust)
    rows, cols = [s[0] for s in shapes], [s[1] for s in shapes]
    ws = space(rr, rows, cols)
    for step in range(2):
        grads = [(torch.randn(s, generator=g, **CUDA) * 1e-3).to(TORCH[gdt]) for s in shapes]
        want = [muon_want(p, gr, mm, None if master is None else master[i], s, hyper, scale)
                for i, (p, gr, mm, s) in enumerate(zip(params, grads, m, shapes))]
        rr.rr_muon(params, grads, m, master, rows, cols, pdt, gdt, hyper, COEFS, scale, ws, ws.numel())
        for i, s in enumerate(shapes):
            new, mom, off = want[i]
            # two products and a sum, each rounded once; the gradient's scale once more
            assert bool(((m[i].double() - mom).abs() <= 6 * U24 * (mom.abs() + 1e-3 * 0.1)).all())
            got = (params if master is None else master)[i].double()
            unit = U[pdt] if master is None else U24
            room = 10 * off / (s[0] * s[1]) ** 0.5 + (3 * U24 + unit) * (new.abs() + 1e-2)
            assert bool(((got - new).abs() <= room).all()), (s, float(((got - new).abs() / room).max()))
            if master is not None:
                assert torch.equal(params[i], master[i].to(TORCH[pdt]))


def test_muon_without_momentum_is_the_orthogonalised_gradient(rr):
    x = matrix((64, 96), seed=2)
    y, = orthogonalize(rr, [x])
    p, m = torch.zeros_like(x), torch.zeros_like(x)
    hyper = rr.rr_muon_hyper(1.0, 0.0, 0.0, 1e-7, 0, rr.RR_MUON_SPECTRAL)
    ws = space(rr, [64], [96])
    rr.rr_muon([p], [x], [m], None, [64], [96], "fp32", "fp32", hyper, COEFS, None, ws, ws.numel())
    assert torch.equal(p, -y) and torch.equal(m, x)


def test_muon_skips_a_step_whose_scale_is_nan(rr):
    shapes = [(40, 70), (300, 280)]
    params, master, m = ([matrix(s, seed=k + 9 * j) for k, s in enumerate(shapes)] for j in range(3))
    grads = [matrix(s, seed=50) for s in shapes]
    before = [t.clone() for t in params + master + m]
    rows, cols = zip(*shapes)
    ws = space(rr, rows, cols)
    scale = torch.full((1,), float("nan"), **CUDA)
    rr.rr_muon(params, grads, m, master, list(rows), list(cols), "fp32", "fp32", rr.rr_muon_hyper(0.1, 0.9, 0.1, 1e-7, 1, 0),
               COEFS, scale, ws, ws.numel())
    assert all(torch.equal(a, b) for a, b in zip(before, params + master + m))


def test_streams_and_graphs(rr):
    shapes = [(200, 300), (513, 129)]
    rows, cols = [s[0] for s in shapes], [s[1] for s in shapes]
    xs = [matrix(s, seed=5) for s in shapes]
    want = orthogonalize(rr, xs)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(x) for x in xs] for _ in streams]
    spaces = [space(rr, rows, cols) for _ in streams]
    torch.cuda.synchronize()
    for s, o, w in zip(streams, outs, spaces):
        with torch.cuda.stream(s):
            for _ in range(4):
                rr.rr_orthogonalize(xs, o, rows, cols, "fp32", "fp32", COEFS, 1e-7, w, w.numel())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))

    p, m = [torch.zeros_like(x) for x in xs], [torch.zeros_like(x) for x in xs]
    grads = [torch.zeros_like(x) for x in xs]
    hyper = rr.rr_muon_hyper(1.0, 0.0, 0.0, 1e-7, 0, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rr.rr_muon(p, grads, m, None, rows, cols, "fp32", "fp32", hyper, COEFS, None, spaces[0], spaces[0].numel())
    for g, x in zip(grads, xs):
        g.copy_(x)
    graph.replay()
    for k, y in enumerate(want):
        f = max(1.0, rows[k] / cols[k]) ** 0.5
        assert bool(((p[k] + y * f).abs() <= 2 * U24 * (y * f).abs()).all())


def test_past_32_bits(rr):
    """A matrix of more than 2^31 elements; its first, middle and last rows against 64 bits."""
    m, n = 33000, 66000
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty((m, n), **CUDA, dtype=torch.bfloat16)
    for at in range(0, m, 3000):
        x[at:at + 3000] = torch.randn((min(3000, m - at), n), generator=g, **CUDA).bfloat16()
    y = torch.empty_like(x)
    coefs = [(3.4445, -4.7750, 2.0315)]
    ws = space(rr, [m], [n])
    rr.rr_orthogonalize([x], [y], [m], [n], "bf16", "bf16", coefs, 1e-7, ws, ws.numel())
    norm = math.sqrt(sum(float(x[k:k + 3000].float().square().sum(dtype=torch.float64)) for k in range(0, m, 3000)))
    pick = [0, 1, 127, 128, 16499, 32512, 32767, 32999]
    part = [x[k:k + 3000] for k in range(0, m, 3000)]

    def times(v, transposed):  # v @ X' or v @ X in 64 bits, a stretch of X at a time
        if transposed:
            return torch.cat([v @ q.double().t() for q in part], 1) / norm
        return sum(v[:, k * 3000:k * 3000 + q.shape[0]] @ q.double() for k, q in enumerate(part)) / norm

    rows = x[pick].double() / norm
    a = times(rows, True)                              # A's rows
    poly = coefs[0][1] * a + coefs[0][2] * times(times(a, False), True)
    for k, i in enumerate(pick):
        poly[k, i] += coefs[0][0]
    want = times(poly, False)
    # one step: no amplification beyond the polynomial's own size, every product within 2^-20
    near(y[pick], want, 2.0 ** -16, U["bf16"])


def test_empty_reference_is_consistent():
    """The 64-bit products agree with the polynomial of the singular values."""
    x = torch.randn(20, 30, dtype=torch.float64)
    u, s, v = torch.linalg.svd(x / (x.norm() + 1e-7), full_matrices=False)
    for a, b, c in COEFS:
        s = s * (a + b * s ** 2 + c * s ** 4)
    assert torch.allclose(products(x, COEFS), u @ torch.diag(s) @ v, rtol=0, atol=1e-10)
