"""rr_layer_norm and rr_layer_norm_backward against the formulas in 64 bits.

Tolerances are bounds on the rounding errors, derived before the first run.
u is the rounding unit of the output's type, e = 2^-24 that of binary32.  A
sum of a row goes through at most D = 80 + cols / 1024 additions in sequence
(32 to a lane, 5 of a warp, 32 warps; for rows too long for registers at least
512 threads have them, which D covers up to 60000 columns), so its error is at most D e times the sum of
magnitudes; a sum over rows through at most R = 100 + rows / 100 (a block has
at most rows / 152 rows, the joins add 8 warps, 38 partials and 16 warps).
"""
import pytest
import torch

from step_util import TINY, TORCH, U, U24, Guarded, generator, guarded_like, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA GPU")
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    return m


def depth(cols):
    return 80 + cols / 1024


def make_x(rows, cols, dtype, seed, offset=0.5, wide=0, shift=0):
    g = generator(seed)
    x = torch.randn((rows, cols + wide), generator=g, device="cuda")
    x *= torch.rand((rows, 1), generator=g, device="cuda") * 2 + 0.25
    x += offset * torch.randn((rows, 1), generator=g, device="cuda")
    buf = guarded_like(x, TORCH[dtype], shift)
    return buf.t.view(rows, cols + wide)[:, :cols]


def make_vec(cols, dtype, seed, base):
    g = generator(seed)
    return (base + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(TORCH[dtype])


def forward_want(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    rstd = (var + eps).rsqrt()
    xhat = (x - mean[:, None]) * rstd[:, None]
    wd = torch.ones_like(x[0]) if w is None else w.double()
    bd = torch.zeros_like(x[0]) if b is None else b.double()
    return xhat * wd + bd, mean, rstd, xhat, wd, bd


def check_forward(x, w, b, eps, y, mean, rstd, dtype, what):
    want, m, r, xhat, wd, bd = forward_want(x, w, b, eps)
    cols = x.shape[1]
    d = depth(cols) + 4
    scale = x.double().abs().mean(1)
    mean_tol = d * U24 * scale + U24 * m.abs()
    shift = mean_tol * r                    # error of the mean in standard deviations
    rstd_rel = d * U24 + shift.square()     # squares are centred: the mean's error enters squared
    tol = (U[dtype] * want.abs() + TINY[dtype]
           + (mean_tol[:, None] + U24 * (x.double() - m[:, None]).abs()) * r[:, None] * wd.abs()
           + (rstd_rel[:, None] + 8 * U24) * (xhat * wd).abs() + 2 * U24 * bd.abs())
    within(y, want, tol * (1 + U[dtype]), f"{what} y")
    if mean is not None:
        within(mean, m, mean_tol + 1e-45, f"{what} mean")
    if rstd is not None:
        within(rstd, r, (rstd_rel + 4 * U24) * r, f"{what} rstd")


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 8), (40, 31), (1, 64), (153, 64), (9, 255), (2000, 256), (7, 257), (1300, 512),
          (160, 513), (33, 1000), (1217, 1024), (5, 1027), (300, 1027), (1, 3584), (8, 3584), (700, 3584), (155, 8192),
          (4, 8193), (160, 8200), (3, 16384), (2, 16385), (3, 18944), (2, 40001), (400, 18944), (330, 9001), (170, 20003),
          (90, 32768), (160, 32776),
          (200, 5120), (180, 6150), (700, 18944), (609, 24576), (620, 9008), (650, 16384)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_forward(rr, rows, cols, dtype, wdtype):
    x = make_x(rows, cols, dtype, rows * 7 + cols)
    w, b = make_vec(cols, wdtype, 1, 1.0), make_vec(cols, wdtype, 2, 0.0)
    y = Guarded(rows * cols, TORCH[dtype])
    mean, rstd = Guarded(rows, torch.float32), Guarded(rows, torch.float32)
    rr.rr_layer_norm(x, w, b, y.t, mean.t, rstd.t, rows, cols, cols, cols, 1e-5, dtype, wdtype)
    check_forward(x, w, b, 1e-5, y.t.view(rows, cols), mean.t, rstd.t, dtype, f"{rows}x{cols}")
    for g in (y, mean, rstd):
        g.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shift,wide", [(1, 0), (0, 3), (0, 8), (3, 5)])
@pytest.mark.parametrize("rows,cols", [(37, 96), (300, 1024), (9, 3584), (200, 2056), (2, 17000)])
def test_forward_strided_and_misaligned(rr, rows, cols, dtype, shift, wide):
    x = make_x(rows, cols, dtype, 5, wide=wide, shift=shift)
    w = make_vec(cols, dtype, 3, 1.0)
    ys = cols + 2 * wide
    y = Guarded(rows * ys, TORCH[dtype], shift)
    y.t.fill_(7)
    rr.rr_layer_norm(x, w, None, y.t, None, None, rows, cols, x.stride(0), ys, 1e-6, dtype, dtype)
    got = y.t.view(rows, ys)
    check_forward(x, w, None, 1e-6, got[:, :cols], None, None, dtype, "strided")
    assert bool((got[:, cols:] == 7).all()), "columns between rows were written"
    y.check()


def test_forward_without_weight_and_bias_and_other_types(rr):
    rows, cols = 70, 520
    x = make_x(rows, cols, "bf16", 9)
    y = torch.empty_like(x)
    rr.rr_layer_norm(x, None, None, y, None, None, rows, cols, cols, cols, 1e-5, "bf16", "bf16")
    check_forward(x, None, None, 1e-5, y, None, None, "bf16", "plain")
    b = make_vec(cols, "fp16", 4, 0.0)
    rr.rr_layer_norm(x, None, b, y, None, None, rows, cols, cols, cols, 1e-5, "bf16", "fp16")
    check_forward(x, None, b, 1e-5, y, None, None, "bf16", "bias of another type")


@pytest.mark.parametrize("rows,cols", [(17, 100), (400, 1024), (30, 3584), (3, 20000), (200, 24000)])
def test_forward_in_place_and_interleaved(rr, rows, cols):
    x = make_x(rows, cols, "bf16", 11)
    keep = x.clone()
    rr.rr_layer_norm(x, None, None, x, None, None, rows, cols, cols, cols, 1e-5, "bf16", "bf16")
    check_forward(keep, None, None, 1e-5, x, None, None, "bf16", "in place")
    both = torch.empty((rows, 2 * cols), device="cuda", dtype=torch.bfloat16)
    both[:, :cols] = keep
    rr.rr_layer_norm(both, None, None, both[:, cols:], None, None, rows, cols, 2 * cols, 2 * cols, 1e-5, "bf16", "bf16")
    check_forward(keep, None, None, 1e-5, both[:, cols:], None, None, "bf16", "beside its input")
    assert torch.equal(both[:, :cols], keep)


def test_forward_row_read_again_and_again(rr):
    x = make_x(1, 640, "fp32", 12)
    y = torch.empty((50, 640), device="cuda")
    rr.rr_layer_norm(x, None, None, y, None, None, 50, 640, 0, 640, 1e-5, "fp32", "fp32")
    check_forward(x.expand(50, 640), None, None, 1e-5, y, None, None, "fp32", "stride 0")


@pytest.mark.parametrize("cols", [5, 300, 1024, 3584, 17000])
@pytest.mark.parametrize("rows", [4, 900])
def test_forward_special_rows(rr, rows, cols):
    """Constant rows, a mean far above the spread, zeros, and rows with NaN or
    infinity, which must not leak into other rows."""
    x = make_x(rows, cols, "fp32", 13)
    x[0] = 3.25
    x[1] = 1000.0 + 0.01 * torch.randn(cols, device="cuda", generator=generator(2))
    x[2, cols // 2] = float("nan")
    x[3, 0] = float("inf")
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    rr.rr_layer_norm(x, None, None, y, mean, rstd, rows, cols, cols, cols, 1e-5, "fp32", "fp32")
    assert bool(torch.isnan(y[2:4]).all()) and bool(torch.isnan(rstd[2:4]).all())
    ok = [i for i in range(rows) if i not in (2, 3)]
    check_forward(x[ok], None, None, 1e-5, y[ok], mean[ok], rstd[ok], "fp32", "special")


def test_forward_large_offsets(rr):
    """More than 2^31 elements: the last rows lie past 32-bit offsets."""
    rows, cols = 600_011, 3584
    x = torch.empty((rows, cols), device="cuda", dtype=torch.bfloat16)
    x.view(torch.int16).random_(0x3C00, 0x4100, generator=generator(3))
    y = torch.empty_like(x)
    rr.rr_layer_norm(x, None, None, y, None, None, rows, cols, cols, cols, 1e-5, "bf16", "bf16")
    for at in (0, (1 << 31) // cols - 1, rows - 3):
        check_forward(x[at:at + 3], None, None, 1e-5, y[at:at + 3], None, None, "bf16", f"row {at}")


def test_forward_on_a_stream_and_in_a_graph(rr):
    rows, cols = 64, 3584
    w = make_vec(cols, "fp32", 5, 1.0)
    x = make_x(rows, cols, "bf16", 21)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rr.rr_layer_norm(x, w, None, y, None, None, rows, cols, cols, cols, 1e-5, "bf16", "fp32", side)
    for seed in (22, 23):
        x.copy_(make_x(rows, cols, "bf16", seed))
        graph.replay()
        check_forward(x, w, None, 1e-5, y, None, None, "bf16", "replay")
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        y.zero_()
        rr.rr_layer_norm(x, w, None, y, None, None, rows, cols, cols, cols, 1e-5, "bf16", "fp32")
    side.synchronize()
    check_forward(x, w, None, 1e-5, y, None, None, "bf16", "side stream")


# ---------------------------------------------------------------- gradient
def workspace(rr, rows, cols):
    n = rr.rr_layer_norm_backward_workspace(rows, cols)
    return Guarded(n, torch.uint8), n


def backward_want(dy, x, w, mean, rstd):
    dy, x = dy.double(), x.double()
    m, r = mean.double()[:, None], rstd.double()[:, None]
    wd = torch.ones_like(x[0]) if w is None else w.double()
    xhat = (x - m) * r
    wdy = dy * wd
    c1, c2 = wdy.mean(1, keepdim=True), (wdy * xhat).mean(1, keepdim=True)
    return (wdy - c1 - xhat * c2) * r, (dy * xhat).sum(0), dy.sum(0), xhat, wdy, r


def check_backward(dy, x, w, mean, rstd, dx, dw, db, dtype, wdtype, what):
    want, dww, dbw, xhat, wdy, r = backward_want(dy, x, w, mean, rstd)
    rows, cols = x.shape
    d = depth(cols) + 8
    over = 100 + rows / 100 + 8
    if dx is not None:
        tol = U[dtype] * want.abs() + TINY[dtype] + U24 * r.abs() * (
            4 * wdy.abs() + d * wdy.abs().mean(1, keepdim=True)
            + xhat.abs() * ((wdy * xhat).abs().mean(1, keepdim=True) * (d + 12)))
        within(dx, want, tol * (1 + U[dtype]), f"{what} dx")
    if dw is not None:
        tol = U[wdtype] * dww.abs() + TINY[wdtype] + over * U24 * (dy.double() * xhat).abs().sum(0)
        within(dw, dww, tol * (1 + U[wdtype]), f"{what} dweight")
    if db is not None:
        tol = U[wdtype] * dbw.abs() + TINY[wdtype] + over * U24 * dy.double().abs().sum(0)
        within(db, dbw, tol * (1 + U[wdtype]), f"{what} dbias")


def statistics(x, eps=1e-5):
    x = x.double()
    mean = x.mean(1)
    rstd = ((x - mean[:, None]).square().mean(1) + eps).rsqrt()
    return mean.float(), rstd.float()


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_backward(rr, rows, cols, dtype, wdtype):
    x = make_x(rows, cols, dtype, rows * 5 + cols)
    dy = make_x(rows, cols, dtype, rows * 3 + cols + 1, offset=0.1)
    w = make_vec(cols, wdtype, 6, 1.0)
    mean, rstd = statistics(x)
    dx = Guarded(rows * cols, TORCH[dtype])
    dw, db = Guarded(cols, TORCH[wdtype]), Guarded(cols, TORCH[wdtype])
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, w, mean, rstd, dx.t, dw.t, db.t, rows, cols, cols, cols, cols, dtype, wdtype,
                              ws.t, n)
    check_backward(dy, x, w, mean, rstd, dx.t.view(rows, cols), dw.t, db.t, dtype, wdtype, f"{rows}x{cols}")
    for g in (dx, dw, db, ws):
        g.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shift,wide", [(1, 0), (0, 3), (0, 8), (3, 5)])
@pytest.mark.parametrize("rows,cols", [(37, 96), (1400, 1024), (9, 3584), (200, 2056), (2, 9000)])
def test_backward_strided_and_misaligned(rr, rows, cols, dtype, shift, wide):
    x = make_x(rows, cols, dtype, 5, wide=wide, shift=shift)
    dy = make_x(rows, cols, dtype, 6, wide=2 * wide, shift=shift)
    mean, rstd = statistics(x)
    xs = cols + wide
    dx = Guarded(rows * xs, TORCH[dtype], shift)
    dx.t.fill_(7)
    dw, db = Guarded(cols, torch.float32, shift), Guarded(cols, torch.float32, shift)
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, None, mean, rstd, dx.t, dw.t, db.t, rows, cols, dy.stride(0), x.stride(0), xs,
                              dtype, "fp32", ws.t, n)
    got = dx.t.view(rows, xs)
    check_backward(dy, x, None, mean, rstd, got[:, :cols], dw.t, db.t, dtype, "fp32", "strided")
    assert bool((got[:, cols:] == 7).all())
    for g in (dx, dw, db, ws):
        g.check()


@pytest.mark.parametrize("rows,cols", [(40, 200), (1300, 1024), (200, 3584), (6, 9000), (300, 17000), (60, 33000)])
def test_backward_parts_in_place_and_broadcast(rr, rows, cols):
    x = make_x(rows, cols, "bf16", 30)
    dy = make_x(rows, cols, "bf16", 31)
    w = make_vec(cols, "bf16", 7, 1.0)
    mean, rstd = statistics(x)
    ws, n = workspace(rr, rows, cols)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    # only the weight's gradient
    rr.rr_layer_norm_backward(dy, x, w, mean, rstd, None, dw, None, rows, cols, cols, cols, cols, "bf16", "bf16", ws.t, n)
    check_backward(dy, x, w, mean, rstd, None, dw, None, "bf16", "bf16", "dweight alone")
    # only dx, over dy
    over = dy.clone()
    rr.rr_layer_norm_backward(over, x, w, mean, rstd, over, None, None, rows, cols, cols, cols, cols, "bf16", "bf16",
                              ws.t, n)
    check_backward(dy, x, w, mean, rstd, over, None, None, "bf16", "bf16", "dx over dy")
    # dx over x
    over = x.clone()
    rr.rr_layer_norm_backward(dy, over, w, mean, rstd, over, None, db, rows, cols, cols, cols, cols, "bf16", "bf16",
                              ws.t, n)
    check_backward(dy, x, w, mean, rstd, over, None, db, "bf16", "bf16", "dx over x")
    # one row of gradients for every row, as a sum's gradient is
    one = dy[:1].contiguous()
    dx = torch.empty_like(x)
    rr.rr_layer_norm_backward(one, x, w, mean, rstd, dx, dw, db, rows, cols, 0, cols, cols, "bf16", "bf16", ws.t, n)
    check_backward(one.expand(rows, cols), x, w, mean, rstd, dx, dw, db, "bf16", "bf16", "broadcast dy")


def test_backward_of_no_rows_gives_zeros(rr):
    dw, db = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
    rr.rr_layer_norm_backward(None, None, None, None, None, None, dw, db, 0, 100, 100, 100, 100, "bf16", "fp32", None, 0)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    rr.rr_layer_norm(None, None, None, None, None, None, 0, 100, 100, 100, 1e-5, "bf16", "fp32")


@pytest.mark.parametrize("rows,cols", [(5, 33), (6, 1100)])
def test_backward_against_differences(rr, rows, cols):
    """Central differences of sum(dy * y) in 64 bits, along random directions.
    Their truncation is h^2 / 6 times a third derivative; h = 1e-4 leaves it
    under 1e-6 of the value's scale, far above the rounding of 1e-16 / h."""
    g = generator(40)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    dy = torch.randn((rows, cols), generator=g, device="cuda")
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    b = 0.2 * torch.randn(cols, generator=g, device="cuda")
    mean, rstd = statistics(x)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, rows, cols, cols, cols, cols, "fp32", "fp32", ws.t, n)

    def loss(xx, ww, bb):
        m = xx.mean(1, keepdim=True)
        r = ((xx - m).square().mean(1, keepdim=True) + 1e-5).rsqrt()
        return float(((xx - m) * r * ww + bb).mul(dy.double()).sum())

    x, w, b, h = x.double(), w.double(), b.double(), 1e-4
    for k in range(6):
        vx, vw, vb = (torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for t in (x, w, b))
        by_hand = (loss(x + h * vx, w + h * vw, b + h * vb) - loss(x - h * vx, w - h * vw, b - h * vb)) / (2 * h)
        terms = [dx.double() * vx, dw.double() * vw, db.double() * vb]
        got = sum(float(t.sum()) for t in terms)
        scale = sum(float(t.abs().sum()) for t in terms)
        assert abs(got - by_hand) <= 2e-6 * scale + 1e-6 * abs(by_hand), (k, got, by_hand, scale)


def test_backward_rows_with_nan_stay_apart(rr):
    rows, cols = 300, 1024
    x = make_x(rows, cols, "fp32", 50)
    dy = make_x(rows, cols, "fp32", 51)
    mean, rstd = statistics(x)
    dy[7, 3] = float("nan")
    dx = torch.empty_like(x)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, None, mean, rstd, dx, dw, db, rows, cols, cols, cols, cols, "fp32", "fp32", ws.t, n)
    assert bool(torch.isnan(dx[7]).all())
    assert bool(torch.isnan(dw[3])) and int(torch.isnan(dw).sum()) == 1 and int(torch.isnan(db).sum()) == 1
    ok = [i for i in range(rows) if i != 7]
    check_backward(dy[ok], x[ok], None, mean[ok], rstd[ok], dx[ok], None, None, "fp32", "fp32", "other rows")


def test_backward_repeats_bit_for_bit_and_in_a_graph(rr):
    rows, cols = 5000, 2048
    x, dy = make_x(rows, cols, "bf16", 60), make_x(rows, cols, "bf16", 61)
    w = make_vec(cols, "fp32", 8, 1.0)
    mean, rstd = statistics(x)
    ws, n = workspace(rr, rows, cols)

    def outputs():
        return torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)

    def call(o, stream=None):
        rr.rr_layer_norm_backward(dy, x, w, mean, rstd, *o, rows, cols, cols, cols, cols, "bf16", "fp32", ws.t, n, stream)

    first, again, replayed = outputs(), outputs(), outputs()
    call(first)
    ws.t.fill_(255)  # the workspace's content does not matter
    call(again)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(replayed, side)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, again, replayed):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_backward_large_offsets(rr):
    rows, cols = 600_011, 3584
    x = torch.empty((rows, cols), device="cuda", dtype=torch.bfloat16)
    x.view(torch.int16).random_(0x3C00, 0x4100, generator=generator(3))
    dy = torch.zeros_like(x)
    at = [0, (1 << 31) // cols - 1, rows - 3]
    for a in at:
        dy[a:a + 3] = make_x(3, cols, "bf16", a)
    mean = torch.full((rows,), 2.0, device="cuda")
    rstd = torch.full((rows,), 0.5, device="cuda")
    dx = torch.empty_like(x)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, None, mean, rstd, dx, dw, db, rows, cols, cols, cols, cols, "bf16", "fp32", ws.t, n)
    some = torch.tensor([a + k for a in at for k in range(3)], device="cuda")
    check_backward(dy[some], x[some], None, mean[some], rstd[some], dx[some], dw, db, "bf16", "fp32", "sampled rows")
