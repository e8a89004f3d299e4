"""Refusals of the losses over logits that need no GPU: arguments are checked
before any CUDA call, and the message names what was wrong."""
import ctypes

import pytest

OK = 4096  # an address that passes the alignment checks and is never read
M = 1 << 20


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


def logp(rr, **kw):
    a = dict(logits=OK, targets=M, logp=2 * M, lse=3 * M, rows=4, vocab=64, stride=64, inv_t=1.0, dtype="bf16", stream=0)
    a.update(kw)
    rr.rr_token_logp(*a.values())


def back(rr, **kw):
    a = dict(logits=OK, targets=M, lse=2 * M, dlogp=3 * M, dlogits=4 * M, rows=4, vocab=64, stride=64, dstride=64,
             inv_t=1.0, dtype="bf16", stream=0)
    a.update(kw)
    rr.rr_token_logp_backward(*a.values())


def policy(rr, hyper=None, **kw):
    a = dict(logits=OK, targets=M, old=2 * M, ref=3 * M, adv=4 * M, weight=5 * M, loss=6 * M, token=7 * M, logp=8 * M,
             dlogits=9 * M, rows=4, vocab=64, stride=64, dstride=64,
             hyper=rr.rr_policy_hyper(*(hyper or (0.2, 0.2, 0.1, 1.0, 1.0))), dtype="bf16", stream=0)
    a.update(kw)
    rr.rr_policy_loss(*a.values())


def preference(rr, hyper=None, **kw):
    a = dict(logits=OK, targets=M, offsets=2 * M, ref=3 * M, loss=4 * M, seq=5 * M, logp=6 * M, dlogits=7 * M, rows=4,
             vocab=64, stride=64, dstride=64, pairs=1,
             hyper=rr.rr_preference_hyper(*(hyper or (0.1, 0.0, 0.0, 1.0, 1.0, 0))), dtype="bf16", workspace=8 * M,
             workspace_bytes=1 << 16, stream=0)
    a.update(kw)
    rr.rr_preference_loss(*a.values())


INF, NAN = float("inf"), float("nan")
ROWS = [
    ("RR_ERR_UNSUPPORTED_DTYPE", "dtype", dict(dtype="int32")),
    ("RR_ERR_UNSUPPORTED_DTYPE", "dtype", dict(dtype=9)),
    ("RR_ERR_INVALID_ARG", "rows", dict(rows=-1)),
    ("RR_ERR_INVALID_ARG", "vocab", dict(vocab=0)),
    ("RR_ERR_INVALID_ARG", "vocab", dict(vocab=(1 << 31) + 1)),
    ("RR_ERR_INVALID_ARG", "logits_stride", dict(stride=63)),
    ("RR_ERR_INVALID_ARG", "logits_stride", dict(rows=1 << 40, stride=1 << 30)),
    ("RR_ERR_INVALID_ARG", "logits is NULL", dict(logits=None)),
    ("RR_ERR_INVALID_ARG", "targets is NULL", dict(targets=None)),
    ("RR_ERR_ALIGNMENT", "logits not", dict(logits=OK + 1)),
    ("RR_ERR_ALIGNMENT", "targets not", dict(targets=M + 4)),
]
TEMPERATURE = [("RR_ERR_INVALID_ARG", "inv_temperature", dict(inv_t=v)) for v in (0.0, -1.0, INF, NAN)]


@pytest.mark.parametrize("status,text,kw", ROWS + TEMPERATURE + [
    ("RR_ERR_INVALID_ARG", "logp is NULL", dict(logp=None)),
    ("RR_ERR_ALIGNMENT", "lse not", dict(lse=3 * M + 2)),
    ("RR_ERR_ALIAS", "logp overlaps logits", dict(logp=OK + 8)),
    ("RR_ERR_ALIAS", "lse overlaps targets", dict(lse=M + 8)),
    ("RR_ERR_ALIAS", "lse overlaps logp", dict(lse=2 * M)),
])
def test_logp_refusals(rr, status, text, kw):
    refused(rr, status, text, lambda: logp(rr, **kw))


@pytest.mark.parametrize("status,text,kw", ROWS + TEMPERATURE + [
    ("RR_ERR_INVALID_ARG", "lse is NULL", dict(lse=None)),
    ("RR_ERR_INVALID_ARG", "dlogp is NULL", dict(dlogp=None)),
    ("RR_ERR_INVALID_ARG", "dlogits is NULL", dict(dlogits=None)),
    ("RR_ERR_INVALID_ARG", "dlogits_stride", dict(dstride=63)),
    ("RR_ERR_ALIGNMENT", "dlogits not", dict(dlogits=4 * M + 1)),
    ("RR_ERR_ALIAS", "dlogits overlaps logits", dict(dlogits=OK + 2)),
    ("RR_ERR_ALIAS", "dlogits overlaps logits", dict(dlogits=OK, dstride=65)),
    ("RR_ERR_ALIAS", "dlogits overlaps lse", dict(dlogits=2 * M)),
])
def test_logp_backward_refusals(rr, status, text, kw):
    refused(rr, status, text, lambda: back(rr, **kw))


@pytest.mark.parametrize("status,text,kw", ROWS + [
    ("RR_ERR_INVALID_ARG", "inv_temperature", dict(hyper=(0.2, 0.2, 0.1, 0.0, 1.0))),
    ("RR_ERR_INVALID_ARG", "inv_temperature", dict(hyper=(0.2, 0.2, 0.1, 1e-60, 1.0))),
    ("RR_ERR_INVALID_ARG", "clip_low", dict(hyper=(-0.1, 0.2, 0.1, 1.0, 1.0))),
    ("RR_ERR_INVALID_ARG", "clip_high", dict(hyper=(0.1, NAN, 0.1, 1.0, 1.0))),
    ("RR_ERR_INVALID_ARG", "kl_coef", dict(hyper=(0.1, 0.2, INF, 1.0, 1.0))),
    ("RR_ERR_INVALID_ARG", "grad_scale", dict(hyper=(0.1, 0.2, 0.1, 1.0, 1e39))),
    ("RR_ERR_INVALID_ARG", "advantages is NULL", dict(adv=None)),
    ("RR_ERR_INVALID_ARG", "token_loss is NULL", dict(token=None)),
    ("RR_ERR_INVALID_ARG", "logp is NULL", dict(logp=None)),
    ("RR_ERR_INVALID_ARG", "dlogits_stride", dict(dstride=1)),
    ("RR_ERR_ALIGNMENT", "loss not", dict(loss=6 * M + 1)),
    ("RR_ERR_ALIGNMENT", "weights not", dict(weight=5 * M + 2)),
    ("RR_ERR_ALIAS", "dlogits overlaps logits", dict(dlogits=OK + 256)),
    ("RR_ERR_ALIAS", "token_loss overlaps dlogits", dict(token=9 * M + 64)),
    ("RR_ERR_ALIAS", "logp overlaps old_logp", dict(logp=2 * M)),
    ("RR_ERR_ALIAS", "token_loss overlaps loss", dict(loss=7 * M)),
    ("RR_ERR_ALIAS", "dlogits overlaps targets", dict(dlogits=M)),
])
def test_policy_refusals(rr, status, text, kw):
    refused(rr, status, text, lambda: policy(rr, **kw))


@pytest.mark.parametrize("status,text,kw", ROWS + [
    ("RR_ERR_INVALID_ARG", "pairs", dict(pairs=0)),
    ("RR_ERR_INVALID_ARG", "pairs", dict(pairs=(1 << 24) + 1)),
    ("RR_ERR_INVALID_ARG", "inv_temperature", dict(hyper=(0.1, 0.0, 0.0, -1.0, 1.0, 0))),
    ("RR_ERR_INVALID_ARG", "beta", dict(hyper=(NAN, 0.0, 0.0, 1.0, 1.0, 0))),
    ("RR_ERR_INVALID_ARG", "label_smoothing", dict(hyper=(0.1, 1.5, 0.0, 1.0, 1.0, 0))),
    ("RR_ERR_INVALID_ARG", "margin", dict(hyper=(0.1, 0.0, INF, 1.0, 1.0, 0))),
    ("RR_ERR_INVALID_ARG", "grad_scale", dict(hyper=(0.1, 0.0, 0.0, 1.0, NAN, 0))),
    ("RR_ERR_INVALID_ARG", "offsets is NULL", dict(offsets=None)),
    ("RR_ERR_INVALID_ARG", "loss is NULL", dict(loss=None)),
    ("RR_ERR_INVALID_ARG", "seq_logp is NULL", dict(seq=None)),
    ("RR_ERR_INVALID_ARG", "logp is NULL", dict(logp=None)),
    ("RR_ERR_INVALID_ARG", "workspace is NULL", dict(workspace=None)),
    ("RR_ERR_INVALID_ARG", "workspace of 8 bytes", dict(workspace_bytes=8)),
    ("RR_ERR_ALIGNMENT", "workspace", dict(workspace=8 * M + 8)),
    ("RR_ERR_ALIGNMENT", "offsets not", dict(offsets=2 * M + 4)),
    ("RR_ERR_ALIAS", "dlogits overlaps logits", dict(dlogits=OK + 256)),
    ("RR_ERR_ALIAS", "logp overlaps seq_logp", dict(logp=5 * M)),
    ("RR_ERR_ALIAS", "workspace overlaps logits", dict(workspace=OK + 64)),
    ("RR_ERR_ALIAS", "seq_logp overlaps offsets", dict(seq=2 * M + 8)),
    ("RR_ERR_ALIAS", "dlogits overlaps ref_logp", dict(dlogits=3 * M)),
])
def test_preference_refusals(rr, status, text, kw):
    refused(rr, status, text, lambda: preference(rr, **kw))


def test_workspaces_and_missing_hypers(rr):
    assert 0 < rr.rr_preference_loss_workspace(0, 1) < rr.rr_preference_loss_workspace(1000, 4)
    for rows, pairs, text in ((-1, 1, "rows"), (1, 0, "pairs")):
        refused(rr, "RR_ERR_INVALID_ARG", text, lambda: rr.rr_preference_loss_workspace(rows, pairs))
    assert rr.lib().rr_preference_loss_workspace(1, 1, None) == rr.RR_ERR_INVALID_ARG
    none = ctypes.POINTER(rr.rr_policy_hyper)()
    refused(rr, "RR_ERR_INVALID_ARG", "hyper is NULL", lambda: rr.rr_policy_loss(
        OK, M, None, None, M, None, None, M, M, None, 1, 8, 8, 8, none, "bf16", 0))
    none = ctypes.POINTER(rr.rr_preference_hyper)()
    refused(rr, "RR_ERR_INVALID_ARG", "hyper is NULL", lambda: rr.rr_preference_loss(
        OK, M, M, None, M, M, M, None, 1, 8, 8, 8, 1, none, "bf16", M, 64, 0))
