"""What the binding of the losses and of Muon refuses without a GPU: tensors that
are not on the device, lists of other lengths."""
import pytest
import torch


@pytest.fixture(scope="module")
def rr():
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    return m


class Elsewhere:
    """A buffer of device 1 where the current one is 0."""

    def get_device(self):
        return 1

    def data_ptr(self):
        return 1 << 20


M = 1 << 20


def calls(rr, x):
    coefs = [(1.5, -0.5, 0.0)]
    return [
        lambda: rr.rr_token_logp(x, M, M, None, 1, 8, 8, 1.0, "fp32", 0),
        lambda: rr.rr_token_logp_backward(M, M, M, M, x, 1, 8, 8, 8, 1.0, "fp32", 0),
        lambda: rr.rr_policy_loss(M, M, None, None, x, None, None, M, M, None, 1, 8, 8, 8,
                                  rr.rr_policy_hyper(0.2, 0.2, 0.0, 1.0, 1.0), "fp32", 0),
        lambda: rr.rr_preference_loss(M, M, x, None, M, M, M, None, 1, 8, 8, 8, 1,
                                      rr.rr_preference_hyper(0.1, 0.0, 0.0, 1.0, 1.0, 0), "fp32", M, 1 << 10, 0),
        lambda: rr.rr_orthogonalize([x], [M], [4], [4], "fp32", "fp32", coefs, 1e-7, M, 1 << 20, 0),
        lambda: rr.rr_muon([M], [2 * M], [x], None, [4], [4], "fp32", "fp32", rr.rr_muon_hyper(0.1, 0.9, 0.0, 1e-7, 1, 0),
                           coefs, None, M, 1 << 20, 0),
    ]


@pytest.mark.parametrize("k", range(6))
def test_tensors_elsewhere(rr, k, monkeypatch):
    from allgather_rr_allreduce_gb300 import _binding
    with pytest.raises(ValueError, match="CUDA tensors"):
        calls(rr, torch.zeros(16))[k]()
    monkeypatch.setattr(_binding, "_device", lambda: 0)
    monkeypatch.setattr(_binding, "_current", None)
    with pytest.raises(rr.RRError) as e:
        calls(rr, Elsewhere())[k]()
    assert e.value.status == rr.RR_ERR_WRONG_DEVICE
