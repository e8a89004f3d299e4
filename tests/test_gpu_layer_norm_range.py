"""rr_layer_norm_backward where 1 / spread^2 or gradient / spread leave
binary32's range and the results do not.

Tolerances as in test_gpu_layer_norm.py (roundings of e = 2^-24 relative, sums of
depth D and R), and for results that may themselves be subnormal four roundings
to binary32's smallest spacing: of the two row means' factors (one of them
times xhat) and of the two sums that make dx.
"""
import pytest
import torch

from step_util import TINY, TORCH, U, U24, Guarded, generator, within
from test_gpu_layer_norm import backward_want, depth, make_vec, rr, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(40, 31), (64, 64), (40, 300), (40, 301), (300, 1024), (1300, 1024), (5, 3584), (200, 2056), (700, 3584),
          (160, 5001), (160, 8192), (700, 9008), (700, 9001), (3, 18944), (30, 9001)]


def check(dy, x, w, mean, rstd, dx, dw, db, dtype, what):
    want, dww, dbw, xhat, wdy, r = backward_want(dy, x, w, mean, rstd)
    rows, cols = x.shape
    d, over = depth(cols) + 8, 108 + rows / 100
    tol = U[dtype] * want.abs() + TINY[dtype] + 2.0 ** -150 * (4 + xhat.abs()) + U24 * r.abs() * (
        4 * wdy.abs() + d * wdy.abs().mean(1, keepdim=True)
        + xhat.abs() * ((wdy * xhat).abs().mean(1, keepdim=True) * (d + 12)))
    within(dx, want, tol * (1 + U[dtype]), f"{what} dx")
    within(dw, dww, (U24 * dww.abs() + TINY["fp32"] + over * U24 * (dy.double() * xhat).abs().sum(0)) * (1 + U24), f"{what} dweight")
    within(db, dbw, (U24 * dbw.abs() + TINY["fp32"] + over * U24 * dy.double().abs().sum(0)) * (1 + U24), f"{what} dbias")


def backward(rr, dy, x, w, mean, rstd, dtype):  # noqa: F811
    rows, cols = x.shape
    dx, dw, db = Guarded(rows * cols, TORCH[dtype]), Guarded(cols, torch.float32), Guarded(cols, torch.float32)
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, w, mean, rstd, dx.t, dw.t, db.t, rows, cols, cols, cols, cols, dtype, "fp32",
                              ws.t, n)
    for b in (dx, dw, db, ws):
        b.check()
    return dx.t.view(rows, cols), dw.t, db.t


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("spread,size", [(1e17, 1e-8), (1e-19, 65536.0), (1e20, 1e-22), (1e30, 1.0), (1e-25, 1e-6)])
def test_spreads_far_from_one(rr, rows, cols, dtype, spread, size):  # noqa: F811
    g = generator(rows + cols)
    x = (torch.randn((rows, cols), generator=g, device="cuda") * spread).to(TORCH[dtype])
    dy = (torch.randn((rows, cols), generator=g, device="cuda") * size).to(TORCH[dtype])
    w = make_vec(cols, "fp32", 6, 1.0)
    xd = x.double()
    mean = xd.mean(1).float()
    rstd = (xd - xd.mean(1, keepdim=True)).square().mean(1).rsqrt().float()
    check(dy, x, w, mean, rstd, *backward(rr, dy, x, w, mean, rstd, dtype), dtype, f"{rows}x{cols}")


@pytest.mark.parametrize("rows,cols", [(40, 31), (64, 96), (40, 301), (300, 1000), (5, 3560), (200, 2056), (160, 5001),
                                       (700, 9008), (700, 9001), (30, 9001)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_constant_rows_far_from_zero(rr, rows, cols, dtype):  # noqa: F811
    """Constant rows, whose mean times rstd leaves binary32's range although xhat
    is 0 throughout: what a lane holds past the row's end must not show."""
    g = generator(rows)
    x = torch.empty((rows, cols), device="cuda", dtype=TORCH[dtype])
    x.copy_(1e33 * (1 + torch.rand((rows, 1), generator=g, device="cuda")))
    mean, rstd = x[:, 0].float().contiguous(), torch.full((rows,), 1e6, device="cuda")
    dy = (torch.randn((rows, cols), generator=g, device="cuda") * 1e-3).to(TORCH[dtype])
    w = make_vec(cols, "fp32", 6, 1.0)
    check(dy, x, w, mean, rstd, *backward(rr, dy, x, w, mean, rstd, dtype), dtype, f"{rows}x{cols}")
