"""Refusals of rr_orthogonalize and rr_muon that need no GPU: arguments are
checked before any CUDA call, and the message names what was wrong."""
import ctypes

import pytest

M = 1 << 20
COEFS = [(3.4445, -4.7750, 2.0315)] * 5
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def rr():
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    return m


def refused(rr, status, text, call):
    with pytest.raises(rr.RRError) as e:
        call()
    assert e.value.status == getattr(rr, status), str(e.value)
    assert text in str(e.value), str(e.value)


def orth(rr, **kw):
    a = dict(x=[M, 2 * M], y=[3 * M, 4 * M], rows=[8, 4], cols=[4, 8], x_dtype="bf16", y_dtype="bf16", coefs=COEFS, eps=1e-7,
             workspace=16 * M, workspace_bytes=M, stream=0)
    a.update(kw)
    rr.rr_orthogonalize(*a.values())


def muon(rr, hyper=None, **kw):
    a = dict(params=[M, 2 * M], grads=[3 * M, 4 * M], momentum=[5 * M, 6 * M], master=[7 * M, 8 * M], rows=[8, 4], cols=[4, 8],
             param_dtype="bf16", grad_dtype="bf16", hyper=rr.rr_muon_hyper(*(hyper or (0.1, 0.9, 0.1, 1e-7, 1, 0))),
             coefs=COEFS, grad_scale=9 * M, workspace=16 * M, workspace_bytes=M, stream=0)
    a.update(kw)
    rr.rr_muon(*a.values())


COMMON = [
    ("RR_ERR_INVALID_ARG", "rows[1]", dict(rows=[8, -1])),
    ("RR_ERR_INVALID_ARG", "rows[0]", dict(rows=[(1 << 20) + 1, 4])),
    ("RR_ERR_INVALID_ARG", "cols[1]", dict(cols=[4, -8])),
    ("RR_ERR_INVALID_ARG", "steps 0", dict(coefs=[])),
    ("RR_ERR_INVALID_ARG", "steps 65", dict(coefs=COEFS * 13)),
    ("RR_ERR_INVALID_ARG", "coefs[4]", dict(coefs=[(1, 1, 1), (1, NAN, 1)])),
    ("RR_ERR_INVALID_ARG", "coefs[0]", dict(coefs=[(INF, 1, 1)])),
    ("RR_ERR_INVALID_ARG", "workspace is NULL", dict(workspace=None)),
    ("RR_ERR_INVALID_ARG", "workspace of 64 bytes", dict(workspace_bytes=64)),
    ("RR_ERR_ALIGNMENT", "workspace", dict(workspace=16 * M + 8)),
]


@pytest.mark.parametrize("status,text,kw", COMMON + [
    ("RR_ERR_UNSUPPORTED_DTYPE", "x_dtype", dict(x_dtype="int32")),
    ("RR_ERR_UNSUPPORTED_DTYPE", "y_dtype", dict(y_dtype=7)),
    ("RR_ERR_INVALID_ARG", "eps", dict(eps=-1.0)),
    ("RR_ERR_INVALID_ARG", "eps", dict(eps=NAN)),
    ("RR_ERR_INVALID_ARG", "x[1] is NULL", dict(x=[M, None])),
    ("RR_ERR_INVALID_ARG", "y[0] is NULL", dict(y=[None, M])),
    ("RR_ERR_ALIGNMENT", "x[0]", dict(x=[M + 1, 2 * M])),
    ("RR_ERR_ALIGNMENT", "y[1]", dict(y=[3 * M, 4 * M + 2], y_dtype="fp32")),
    ("RR_ERR_ALIAS", "overlaps", dict(y=[M + 2, 4 * M])),
    ("RR_ERR_ALIAS", "overlaps", dict(y=[2 * M, 4 * M])),
    ("RR_ERR_ALIAS", "overlaps", dict(y=[M, 4 * M], y_dtype="fp32")),
    ("RR_ERR_ALIAS", "overlaps", dict(y=[3 * M, 3 * M])),
    ("RR_ERR_ALIAS", "overlaps", dict(y=[3 * M, 16 * M])),
])
def test_orthogonalize_refusals(rr, status, text, kw):
    refused(rr, status, text, lambda: orth(rr, **kw))


@pytest.mark.parametrize("status,text,kw", COMMON + [
    ("RR_ERR_UNSUPPORTED_DTYPE", "param_dtype", dict(param_dtype="int32")),
    ("RR_ERR_UNSUPPORTED_DTYPE", "grad_dtype", dict(grad_dtype="int32")),
    ("RR_ERR_INVALID_ARG", "lr", dict(hyper=(-0.1, 0.9, 0.1, 1e-7, 1, 0))),
    ("RR_ERR_INVALID_ARG", "momentum", dict(hyper=(0.1, 1.0, 0.1, 1e-7, 1, 0))),
    ("RR_ERR_INVALID_ARG", "weight_decay", dict(hyper=(0.1, 0.9, NAN, 1e-7, 1, 0))),
    ("RR_ERR_INVALID_ARG", "eps", dict(hyper=(0.1, 0.9, 0.1, -1.0, 1, 0))),
    ("RR_ERR_INVALID_ARG", "adjust", dict(hyper=(0.1, 0.9, 0.1, 1e-7, 1, 2))),
    ("RR_ERR_INVALID_ARG", "momentum[1] is NULL", dict(momentum=[5 * M, None])),
    ("RR_ERR_INVALID_ARG", "master[0] is NULL", dict(master=[None, 8 * M])),
    ("RR_ERR_ALIGNMENT", "grads[0]", dict(grads=[3 * M + 1, 4 * M])),
    ("RR_ERR_ALIGNMENT", "momentum[0]", dict(momentum=[5 * M + 2, 6 * M])),
    ("RR_ERR_ALIGNMENT", "grad_scale", dict(grad_scale=9 * M + 2)),
    ("RR_ERR_ALIAS", "overlaps", dict(grads=[M, 4 * M])),
    ("RR_ERR_ALIAS", "overlaps", dict(momentum=[5 * M, 5 * M + 64])),
    ("RR_ERR_ALIAS", "overlaps", dict(grad_scale=5 * M)),
    ("RR_ERR_ALIAS", "overlaps", dict(workspace=7 * M)),
])
def test_muon_refusals(rr, status, text, kw):
    refused(rr, status, text, lambda: muon(rr, **kw))


def test_workspace_and_lists(rr):
    assert rr.rr_orthogonalize_workspace([], []) == 0
    assert rr.rr_orthogonalize_workspace([0, 5], [7, 0]) == 0
    one = rr.rr_orthogonalize_workspace([100], [200])
    assert one > 0 and one == rr.rr_orthogonalize_workspace([200], [100])
    assert rr.rr_orthogonalize_workspace([100, 100], [200, 200]) == 2 * one
    refused(rr, "RR_ERR_INVALID_ARG", "rows[0]", lambda: rr.rr_orthogonalize_workspace([-1], [4]))
    assert rr.lib().rr_orthogonalize_workspace(None, None, 0, None) == rr.RR_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        rr.rr_orthogonalize_workspace([1, 2], [3])
    with pytest.raises(ValueError):
        orth(rr, coefs=[(1, 2)])
    with pytest.raises(ValueError):
        orth(rr, x=[M])
    refused(rr, "RR_ERR_INVALID_ARG", "hyper is NULL", lambda: rr.rr_muon(
        [M], [2 * M], [3 * M], None, [4], [4], "bf16", "bf16", ctypes.POINTER(rr.rr_muon_hyper)(), COEFS, None, 16 * M, M, 0))
