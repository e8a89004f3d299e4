"""What rr_layer_norm_backward_workspace asks for: room for what the kernels
keep, and not many times that."""
import pytest


@pytest.fixture(scope="module")
def rr():
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    return m


@pytest.mark.parametrize("rows,cols,partials", [
    (4096, 18944, 152),       # a block of the one-pass kernel to each SM
    (608, 24576, 152), (100, 18944, 100), (100_000, 8193, 152),
    (4096, 24577, 19), (4096, 131072, 4), (1024, 1 << 20, 1), (1 << 20, 1 << 22, 1), (3, 1 << 31, 1),
    (100_000, 8192, 608), (10, 64, 10),
])
def test_partial_sums(rr, rows, cols, partials):
    """Two sums of `cols` binary32 for each partial, and 8 bytes a row."""
    got = rr.rr_layer_norm_backward_workspace(rows, cols)
    most = 8 * rows + 16 + 2 * 4 * cols * partials
    assert got <= most, (got, most)
    assert got >= 8 * rows + 2 * 4 * cols * min(rows, 1)
