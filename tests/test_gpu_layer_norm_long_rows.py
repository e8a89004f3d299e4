"""Layer norm of rows of millions of columns: the rounding of a row's sums
does not grow with its length.

A thread adds at most 64 values in binary32 before a compensated sum takes over,
whose own rounding is one of the result's; then 5 additions of a warp, 32 of the
block's warps, and a few roundings of the values themselves: D = 112 roundings of
e = 2^-24 relative to the sum of magnitudes, whatever the length.  The data is
nearly constant, so that roundings of a long sum in sequence would add up.
"""
import pytest
import torch

from step_util import U24, Guarded, generator, within
from test_gpu_layer_norm import backward_want, forward_want, rr, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

D = 112
LONG = [1 << 24, (1 << 24) + 3]


def nearly(value, rows, cols, seed):
    return value + torch.randn((rows, cols), generator=generator(seed), device="cuda") * 2.0 ** -10


@pytest.mark.parametrize("cols", LONG)
def test_forward(rr, cols):  # noqa: F811
    rows = 2
    x = nearly(1.1, rows, cols, 1)
    y, mean, rstd = (Guarded(n, torch.float32) for n in (rows * cols, rows, rows))
    rr.rr_layer_norm(x, None, None, y.t, mean.t, rstd.t, rows, cols, cols, cols, 1e-5, "fp32", "fp32")
    want, m, r, xhat, _, _ = forward_want(x, None, None, 1e-5)
    mean_tol = (D * x.double().abs().mean(1) + m.abs()) * U24
    rstd_rel = D * U24 + (mean_tol * r).square()   # squares are centred: the mean's error enters squared
    within(mean.t, m, mean_tol, "mean")
    within(rstd.t, r, (rstd_rel + 4 * U24) * r, "rstd")
    within(y.t.view(rows, cols), want, 2 * U24 * want.abs() + 2.0 ** -149
           + (mean_tol[:, None] + U24 * (x.double() - m[:, None]).abs()) * r[:, None]
           + (rstd_rel[:, None] + 8 * U24) * xhat.abs(), "y")
    for b in (y, mean, rstd):
        b.check()


@pytest.mark.parametrize("cols", LONG)
def test_backward(rr, cols):  # noqa: F811
    rows = 2
    x, dy = nearly(1.1, rows, cols, 2), nearly(1.3, rows, cols, 3)
    mean = x.double().mean(1).float()
    rstd = torch.full((rows,), 500.0, device="cuda")
    dx, dw, db = (Guarded(n, torch.float32) for n in (rows * cols, cols, cols))
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, None, mean, rstd, dx.t, dw.t, db.t, rows, cols, cols, cols, cols, "fp32", "fp32",
                              ws.t, n)
    want, dww, dbw, xhat, wdy, r = backward_want(dy, x, None, mean, rstd)
    tol = U24 * want.abs() + 2.0 ** -149 + U24 * r * (
        4 * wdy.abs() + (D + 8) * wdy.abs().mean(1, keepdim=True)
        + xhat.abs() * ((wdy * xhat).abs().mean(1, keepdim=True) * (D + 20)))
    within(dx.t.view(rows, cols), want, tol * 1.01, "dx")
    within(dw.t, dww, 16 * U24 * (dy.double() * xhat).abs().sum(0), "dweight")
    within(db.t, dbw, 16 * U24 * dy.double().abs().sum(0), "dbias")
    for b in (dx, dw, db, ws):
        b.check()
