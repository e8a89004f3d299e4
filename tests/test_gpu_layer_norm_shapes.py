"""Layer norm and its gradient where blocks and warps work through many rows of
their own: rings and row-ahead registers used again and again, row statistics
fetched 32 rows at a time, long rows of any width in one pass over HBM.  Every row
has statistics of its own; bounds as in test_gpu_layer_norm.py."""
import pytest
import torch

import test_gpu_layer_norm as base
from step_util import TORCH, Guarded, generator
from test_gpu_layer_norm import check_backward, check_forward, make_vec, make_x, rr, statistics, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

MANY = [(65536, 64), (70001, 200), (50000, 300), (50000, 301), (40000, 1000), (30000, 1027), (20000, 3584),
        (9001, 5001), (9000, 6144), (9000, 8192), (12001, 7001)]
WIDE = [(700, 9001), (700, 18945), (700, 24575), (2001, 12001), (3000, 16392), (1300, 20480), (1300, 24576)]
TYPES = [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")]


@pytest.mark.parametrize("rows,cols", MANY + WIDE)
@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_forward(rr, rows, cols, dtype, wdtype):  # noqa: F811
    x = make_x(rows, cols, dtype, rows + cols)
    w, b = make_vec(cols, wdtype, 1, 1.0), make_vec(cols, wdtype, 2, 0.0)
    y, mean, rstd = Guarded(rows * cols, TORCH[dtype]), Guarded(rows, torch.float32), Guarded(rows, torch.float32)
    rr.rr_layer_norm(x, w, b, y.t, mean.t, rstd.t, rows, cols, cols, cols, 1e-5, dtype, wdtype)
    check_forward(x, w, b, 1e-5, y.t.view(rows, cols), mean.t, rstd.t, dtype, f"{rows}x{cols}")
    for g in (y, mean, rstd):
        g.check()


@pytest.mark.parametrize("rows,cols", MANY + WIDE)
@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_backward(rr, rows, cols, dtype, wdtype):  # noqa: F811
    x = make_x(rows, cols, dtype, rows + 2 * cols)
    dy = make_x(rows, cols, dtype, rows + 3 * cols, offset=0.1)
    w = make_vec(cols, wdtype, 6, 1.0)
    mean, rstd = statistics(x)
    dx, dw, db = Guarded(rows * cols, TORCH[dtype]), Guarded(cols, TORCH[wdtype]), Guarded(cols, TORCH[wdtype])
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, w, mean, rstd, dx.t, dw.t, db.t, rows, cols, cols, cols, cols, dtype, wdtype,
                              ws.t, n)
    check_backward(dy, x, w, mean, rstd, dx.t.view(rows, cols), dw.t, db.t, dtype, wdtype, f"{rows}x{cols}")
    for g in (dx, dw, db, ws):
        g.check()


@pytest.mark.parametrize("rows,cols", [(9000, 200), (9000, 301), (9000, 1000), (5000, 3584), (5000, 5001), (700, 9008),
                                       (700, 9001), (1300, 18945), (1300, 24000)])
def test_parts_in_place_and_broadcast(rr, rows, cols):  # noqa: F811
    base.test_backward_parts_in_place_and_broadcast(rr, rows, cols)


@pytest.mark.parametrize("rows,cols", [(9000, 301), (9000, 1000), (5000, 3584), (5000, 5001), (2000, 24001)])
def test_forward_in_place_and_interleaved(rr, rows, cols):  # noqa: F811
    base.test_forward_in_place_and_interleaved(rr, rows, cols)


def test_large_offsets_with_statistics_of_each_row(rr):  # noqa: F811
    """More than 2^31 elements, and no two rows with the same mean and rstd."""
    rows, cols = 600_011, 3584
    x = torch.empty((rows, cols), device="cuda", dtype=torch.bfloat16)
    x.view(torch.int16).random_(0x3C00, 0x4100, generator=generator(3))
    dy = torch.zeros_like(x)
    at = [0, 152 * 32 * 3 - 1, (1 << 31) // cols - 1, rows - 3]
    for a in at:
        dy[a:a + 3] = make_x(3, cols, "bf16", a)
    mean = 1.5 + torch.rand(rows, device="cuda", generator=generator(4))
    rstd = 0.25 + 0.5 * torch.rand(rows, device="cuda", generator=generator(5))
    dx = torch.empty_like(x)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws, n = workspace(rr, rows, cols)
    rr.rr_layer_norm_backward(dy, x, None, mean, rstd, dx, dw, db, rows, cols, cols, cols, cols, "bf16", "fp32", ws.t, n)
    some = torch.tensor([a + k for a in at for k in range(3)], device="cuda")
    check_backward(dy[some], x[some], None, mean[some], rstd[some], dx[some], dw, db, "bf16", "fp32", "sampled rows")
    ws.check()
