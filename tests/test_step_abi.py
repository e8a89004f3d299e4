"""Refusals of the training-step operators that need no GPU: arguments are
checked before any CUDA call, and the message names what was wrong."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK = 4096  # an address that passes the alignment checks and is never read


@pytest.fixture(scope="module")
def rr():
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    return m


def refused(rr, status, text, call, *args):
    with pytest.raises(rr.RRError) as e:
        call(*args)
    assert e.value.status == status, str(e.value)
    assert text in str(e.value), str(e.value)


def norm(rr, **kw):
    a = dict(x=OK, weight=None, bias=None, y=1 << 20, mean=None, rstd=None, rows=4, cols=64, x_stride=64, y_stride=64,
             eps=1e-5, dtype="bf16", weight_dtype="bf16", stream=0)
    a.update(kw)
    rr.rr_layer_norm(*a.values())


def grad(rr, **kw):
    a = dict(dy=OK, x=1 << 20, weight=None, mean=1 << 21, rstd=1 << 22, dx=1 << 23, dweight=1 << 24, dbias=1 << 25,
             rows=4, cols=64, dy_stride=64, x_stride=64, dx_stride=64, dtype="bf16", weight_dtype="bf16",
             workspace=1 << 26, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    rr.rr_layer_norm_backward(*a.values())


@pytest.mark.parametrize("status,text,kw", [
    ("RR_ERR_UNSUPPORTED_DTYPE", "dtype", dict(dtype="int32")),
    ("RR_ERR_UNSUPPORTED_DTYPE", "weight_dtype", dict(weight_dtype="int32")),
    ("RR_ERR_UNSUPPORTED_DTYPE", "dtype", dict(dtype=9)),
    ("RR_ERR_INVALID_ARG", "rows", dict(rows=-1)),
    ("RR_ERR_INVALID_ARG", "cols", dict(cols=0)),
    ("RR_ERR_INVALID_ARG", "cols", dict(cols=(1 << 31) + 1)),
    ("RR_ERR_INVALID_ARG", "x_stride", dict(x_stride=-64)),
    ("RR_ERR_INVALID_ARG", "y_stride", dict(y_stride=63)),
    ("RR_ERR_INVALID_ARG", "eps", dict(eps=-1.0)),
    ("RR_ERR_INVALID_ARG", "eps", dict(eps=float("nan"))),
    ("RR_ERR_INVALID_ARG", "x is NULL", dict(x=None)),
    ("RR_ERR_INVALID_ARG", "y is NULL", dict(y=None)),
    ("RR_ERR_ALIGNMENT", "x not", dict(x=OK + 1)),
    ("RR_ERR_ALIGNMENT", "bias not", dict(bias=(1 << 22) + 2, weight_dtype="fp32")),
    ("RR_ERR_ALIGNMENT", "mean not", dict(mean=(1 << 22) + 2)),
    ("RR_ERR_ALIAS", "y overlaps x", dict(y=OK + 2)),
    ("RR_ERR_ALIAS", "y overlaps x", dict(y=OK, y_stride=128)),
    ("RR_ERR_ALIAS", "y overlaps x", dict(x_stride=128, y_stride=128, y=OK + 63 * 2)),
    ("RR_ERR_ALIAS", "y overlaps", dict(weight=(1 << 20) + 16)),
    ("RR_ERR_ALIAS", "y overlaps", dict(rstd=(1 << 20) + 16)),
    ("RR_ERR_ALIAS", "statistic", dict(mean=OK + 16)),
    ("RR_ERR_ALIAS", "mean overlaps rstd", dict(mean=1 << 22, rstd=(1 << 22) + 4)),
])
def test_layer_norm_refusals(rr, status, text, kw):
    refused(rr, getattr(rr, status), text, lambda: norm(rr, **kw))


@pytest.mark.parametrize("status,text,kw", [
    ("RR_ERR_UNSUPPORTED_DTYPE", "dtype", dict(dtype="int32")),
    ("RR_ERR_INVALID_ARG", "all NULL", dict(dx=None, dweight=None, dbias=None)),
    ("RR_ERR_INVALID_ARG", "dy is NULL", dict(dy=None)),
    ("RR_ERR_INVALID_ARG", "rstd is NULL", dict(rstd=None)),
    ("RR_ERR_INVALID_ARG", "dx_stride", dict(dx_stride=10)),
    ("RR_ERR_INVALID_ARG", "dy_stride", dict(dy_stride=-1)),
    ("RR_ERR_INVALID_ARG", "workspace is NULL", dict(workspace=None)),
    ("RR_ERR_INVALID_ARG", "workspace of 16 bytes", dict(workspace_bytes=16)),
    ("RR_ERR_ALIGNMENT", "workspace", dict(workspace=(1 << 26) + 8)),
    ("RR_ERR_ALIGNMENT", "dbias", dict(dbias=(1 << 25) + 1)),
    ("RR_ERR_ALIAS", "dx overlaps dy", dict(dx=OK + 2)),
    ("RR_ERR_ALIAS", "dx overlaps x", dict(dx=1 << 20, dx_stride=65)),
    ("RR_ERR_ALIAS", "dweight overlaps x", dict(dweight=(1 << 20) + 64)),
    ("RR_ERR_ALIAS", "workspace overlaps mean", dict(workspace=(1 << 21) - 64)),
    ("RR_ERR_ALIAS", "dbias overlaps dweight", dict(dbias=1 << 24)),
    ("RR_ERR_ALIAS", "dbias overlaps dweight", dict(rows=0, dbias=1 << 24)),
])
def test_layer_norm_backward_refusals(rr, status, text, kw):
    refused(rr, getattr(rr, status), text, lambda: grad(rr, **kw))


def test_workspace_sizes(rr):
    assert rr.rr_layer_norm_backward_workspace(0, 64) == 0
    small, big = (rr.rr_layer_norm_backward_workspace(r, 64) for r in (10, 100000))
    assert 0 < small < big
    refused(rr, rr.RR_ERR_INVALID_ARG, "cols", rr.rr_layer_norm_backward_workspace, 1, 0)
    assert rr.rr_grad_norm_workspace(0) > 0
    assert rr.rr_grad_norm_workspace(100000) > rr.rr_grad_norm_workspace(1)
    refused(rr, rr.RR_ERR_INVALID_ARG, "num_tensors", rr.rr_grad_norm_workspace, -1)
    assert rr.lib().rr_grad_norm_workspace(1, None) == rr.RR_ERR_INVALID_ARG
    assert rr.lib().rr_layer_norm_backward_workspace(1, 1, None) == rr.RR_ERR_INVALID_ARG


def gradnorm(rr, **kw):
    a = dict(grads=[OK, 1 << 20], sizes=[8, 8], dtype="bf16", inv_scale=1.0, max_norm=1.0, norm=1 << 21, scale=1 << 22,
             workspace=1 << 23, workspace_bytes=1 << 20, stream=0)
    a.update(kw)
    rr.rr_grad_norm(*a.values())


@pytest.mark.parametrize("status,text,kw", [
    ("RR_ERR_UNSUPPORTED_DTYPE", "dtype", dict(dtype="int32")),
    ("RR_ERR_INVALID_ARG", "sizes[1]", dict(sizes=[8, -1])),
    ("RR_ERR_INVALID_ARG", "grads[1] is NULL", dict(grads=[OK, None])),
    ("RR_ERR_INVALID_ARG", "inv_scale", dict(inv_scale=0.0)),
    ("RR_ERR_INVALID_ARG", "inv_scale", dict(inv_scale=float("nan"))),
    ("RR_ERR_INVALID_ARG", "max_norm", dict(max_norm=-1.0)),
    ("RR_ERR_INVALID_ARG", "max_norm", dict(max_norm=float("nan"))),
    ("RR_ERR_INVALID_ARG", "both NULL", dict(norm=None, scale=None)),
    ("RR_ERR_INVALID_ARG", "workspace is NULL", dict(workspace=None)),
    ("RR_ERR_INVALID_ARG", "needed", dict(workspace_bytes=64)),
    ("RR_ERR_ALIGNMENT", "grads[0]", dict(grads=[OK + 1, 1 << 20])),
    ("RR_ERR_ALIGNMENT", "norm", dict(norm=(1 << 21) + 2)),
    ("RR_ERR_ALIGNMENT", "workspace", dict(workspace=(1 << 23) + 4)),
    ("RR_ERR_ALIAS", "overlaps", dict(norm=1 << 22)),
    ("RR_ERR_ALIAS", "overlaps", dict(scale=OK + 4)),
    ("RR_ERR_ALIAS", "overlaps", dict(workspace=(1 << 20) - 16)),
])
def test_grad_norm_refusals(rr, status, text, kw):
    refused(rr, getattr(rr, status), text, lambda: gradnorm(rr, **kw))


HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1)


def hyper(rr, **kw):
    return rr.rr_adamw_hyper(*{**HYPER, **kw}.values())


def adamw(rr, eight, h=None, **kw):
    a = dict(params=[1 << 20, 2 << 20], grads=[3 << 20, 4 << 20], m=[5 << 20, 6 << 20], ms=[7 << 20, 8 << 20],
             v=[9 << 20, 10 << 20], vs=[11 << 20, 12 << 20], master=[13 << 20, 14 << 20], sizes=[300, 300], pd="bf16",
             gd="bf16", hyper=h or hyper(rr), seed=1, scale=OK, stream=0)
    a.update(kw)
    if eight:
        rr.rr_adamw8(*a.values())
    else:
        for k in ("ms", "vs", "seed"):
            del a[k]
        rr.rr_adamw(*a.values())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("status,text,kw", [
    ("RR_ERR_UNSUPPORTED_DTYPE", "param_dtype", dict(pd="int32")),
    ("RR_ERR_UNSUPPORTED_DTYPE", "grad_dtype", dict(gd=7)),
    ("RR_ERR_INVALID_ARG", "sizes[0]", dict(sizes=[-2, 300])),
    ("RR_ERR_INVALID_ARG", "params[0] is NULL", dict(params=[None, 2 << 20])),
    ("RR_ERR_INVALID_ARG", "exp_avg_sq[1] is NULL", dict(v=[9 << 20, None])),
    ("RR_ERR_INVALID_ARG", "master[1] is NULL", dict(master=[13 << 20, None])),
    ("RR_ERR_ALIGNMENT", "grads[1]", dict(grads=[3 << 20, (4 << 20) + 1])),
    ("RR_ERR_ALIGNMENT", "master[0]", dict(master=[(13 << 20) + 2, 14 << 20])),
    ("RR_ERR_ALIGNMENT", "grad_scale", dict(scale=OK + 2)),
    ("RR_ERR_ALIAS", "overlaps", dict(params=[1 << 20, (1 << 20) + 598])),
    ("RR_ERR_ALIAS", "overlaps", dict(grads=[(1 << 20) + 2, 4 << 20])),
    ("RR_ERR_ALIAS", "overlaps", dict(m=[5 << 20, 5 << 20])),
    ("RR_ERR_ALIAS", "overlaps", dict(scale=1 << 20)),
])
def test_adamw_refusals(rr, eight, status, text, kw):
    refused(rr, getattr(rr, status), text, lambda: adamw(rr, eight, **kw))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("field,value", [("lr", -1.0), ("lr", float("nan")), ("beta1", 1.0), ("beta1", -0.1),
                                         ("beta2", 1.0), ("beta2", float("nan")), ("eps", -1e-8),
                                         ("weight_decay", -0.1), ("step", 0)])
def test_adamw_hyper_refusals(rr, eight, field, value):
    refused(rr, rr.RR_ERR_INVALID_ARG, field, lambda: adamw(rr, eight, hyper(rr, **{field: value})))


def test_adamw8_scale_refusals(rr):
    refused(rr, rr.RR_ERR_INVALID_ARG, "exp_avg_scale[0] is NULL", lambda: adamw(rr, True, ms=[None, 8 << 20]))
    refused(rr, rr.RR_ERR_ALIGNMENT, "exp_avg_sq_scale[1]", lambda: adamw(rr, True, vs=[11 << 20, (12 << 20) + 1]))
    refused(rr, rr.RR_ERR_ALIAS, "overlaps", lambda: adamw(rr, True, vs=[11 << 20, (11 << 20) + 4]))


def test_lists_that_hold_nothing_need_no_gpu(rr):
    """Empty lists and empty tensors return before any CUDA call."""
    adamw(rr, False, params=[], grads=[], m=[], v=[], master=None, sizes=[])
    adamw(rr, True, params=[None], grads=[None], m=[None], ms=[None], v=[None], vs=[None], master=[None], sizes=[0])
    assert rr.lib().rr_adamw(None, None, None, None, None, None, 0, 0, 0, ctypes.byref(hyper(rr)), None, None) == rr.RR_OK
    norm(rr, rows=0, x=None, y=None)


def test_lists_of_unequal_length_are_refused_by_the_binding(rr):
    with pytest.raises(ValueError, match="grads"):
        adamw(rr, False, grads=[OK])


def test_alias_rule_against_every_pair(tmp_path):
    """rr_spans.h compiled for the host and compared with brute force."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = tmp_path / "spans_check"
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "allgather_rr_allreduce_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "native", "spans_check.cpp"), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr
