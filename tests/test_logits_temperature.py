"""Temperatures whose scales leave binary32's range are refused; no GPU needed."""
import pytest

from test_logits_abi import back, logp, policy, preference, refused, rr  # noqa: F401


@pytest.mark.parametrize("inv_t", [3e38, 2.0 ** -121, 1e-44])
def test_extreme_temperatures(rr, inv_t):  # noqa: F811
    for call in (lambda: logp(rr, inv_t=inv_t), lambda: back(rr, inv_t=inv_t),
                 lambda: policy(rr, hyper=(0.2, 0.2, 0.1, inv_t, 1.0)),
                 lambda: preference(rr, hyper=(0.1, 0.0, 0.0, inv_t, 1.0, 0))):
        refused(rr, "RR_ERR_INVALID_ARG", "inv_temperature", call)
