"""The weight's gradient of long rows, many of them: the rounding of a sum over
rows does not grow with their number.

A thread adds at most 64 rows in binary32 before a compensated sum takes over,
whose own rounding is one of the result's; the join adds at most 19 partial sums
in sequence and 5 of a warp, and a product is off by 4 roundings: R = 96
roundings of e = 2^-24 relative to the sum of magnitudes.  dy is nearly constant
and rounds the same way at each addition, so that a long sum in sequence would
add the roundings up.
"""
import pytest
import torch

from step_util import U24, Guarded, generator, within
from test_gpu_layer_norm import rr, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

R = 96


@pytest.mark.parametrize("rows,cols", [(6001, 131072), (6001, 131073), (4500, 26001)])
def test_weight_gradient_of_many_long_rows(rr, rows, cols):  # noqa: F811
    g = generator(rows + cols)
    x = torch.randn((rows, cols), generator=g, device="cuda").abs_()
    dy = torch.full((rows, cols), 1 + 0.45 * 2.0 ** -13 + 2.0 ** -4, device="cuda")
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dw, db = Guarded(cols, torch.float32), Guarded(cols, torch.float32)
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, None, mean, rstd, None, dw.t, db.t, rows, cols, cols, cols, cols, "fp32", "fp32",
                              ws.t, n)
    for at in (0, cols - 2000):
        part = slice(at, at + 2000)
        dyd, xd = dy[:, part].double(), x[:, part].double()
        within(db.t[part], dyd.sum(0), R * U24 * dyd.abs().sum(0), "dbias")
        within(dw.t[part], (dyd * xd).sum(0), R * U24 * (dyd * xd).abs().sum(0), "dweight")
    for b in (dw, db, ws):
        b.check()
