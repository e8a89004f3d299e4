"""A list whose matrices are too large for a call's tables is refused before any
work, wherever they stand in it; no GPU needed (the refusal comes first)."""
import pytest

COEFS = [(3.4445, -4.7750, 2.0315)] * 5
SIDE = 1 << 20  # the largest: 2^27 blocks of 128 x 64, so that 16 in one table pass 2^31 - 1
T = 1 << 44


@pytest.fixture(scope="module")
def rr():
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    return m


def lists(small, large):
    rows = [4] * small + [SIDE] * large
    cols = [8] * small + [SIDE] * large
    return rows, cols


def addresses(n, first):  # 2^44 apart, beyond a matrix of 2^40 binary32 values
    return [(first + k) * T for k in range(n)]


@pytest.mark.parametrize("small,large", [(0, 16), (0, 17), (160, 16), (170, 16), (160, 40), (320, 16)])
def test_refused_before_work(rr, small, large):
    rows, cols = lists(small, large)
    n = len(rows)
    x, y, z = (addresses(n, 1 + k * n) for k in range(3))
    # the workspace behind them: addresses stay below 2^62
    space, size = (1 + 3 * n) * T, 1 << 60
    for call in (
        lambda: rr.rr_orthogonalize_workspace(rows, cols),
        lambda: rr.rr_orthogonalize(x, y, rows, cols, "fp32", "fp32", COEFS, 1e-7, space, size, 0),
        lambda: rr.rr_muon(x, y, z, None, rows, cols, "fp32", "fp32", rr.rr_muon_hyper(0.1, 0.9, 0.0, 1e-7, 1, 0), COEFS,
                           None, space, size, 0),
    ):
        with pytest.raises(rr.RRError) as e:
            call()
        assert e.value.status == rr.RR_ERR_INVALID_ARG and "too large" in str(e.value), str(e.value)


@pytest.mark.parametrize("small,large", [(0, 15), (145, 15), (160, 15)])
def test_as_many_as_fit_have_a_workspace(rr, small, large):
    assert rr.rr_orthogonalize_workspace(*lists(small, large)) >= 15 * 8 * SIDE * SIDE
