"""Tensors of another device than the current one are refused by the binding of
the training-step operators, before the library is called (needs no GPU: the
tensors are stand-ins)."""
import pytest


class Stand:
    """What the binding asks of a torch tensor."""
    is_cuda = True

    def __init__(self, device, address=4096):
        self.device, self.address = device, address

    def get_device(self):
        return self.device

    def data_ptr(self):
        return self.address


@pytest.fixture
def rr(monkeypatch):
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    from allgather_rr_allreduce_gb300 import _binding
    m.lib()
    monkeypatch.setattr(_binding, "_tensor_class", Stand)
    monkeypatch.setattr(_binding, "_device", lambda: 0)
    monkeypatch.setattr(_binding, "_current", None, raising=False)
    return m


def refused(rr, call, *args):
    with pytest.raises(rr.RRError, match="device 1") as e:
        call(*args)
    assert e.value.status == rr.RR_ERR_WRONG_DEVICE


H, T = 0, 1   # here, there


@pytest.mark.parametrize("which", range(6))
def test_layer_norm(rr, which):
    t = [Stand(T if i == which else H, 4096 << i) for i in range(6)]
    refused(rr, rr.rr_layer_norm, *t, 1, 8, 8, 8, 1e-5, "bf16", "bf16", 0)


@pytest.mark.parametrize("which", range(9))
def test_layer_norm_backward(rr, which):
    t = [Stand(T if i == which else H, 4096 << i) for i in range(9)]
    refused(rr, rr.rr_layer_norm_backward, *t[:8], 1, 8, 8, 8, 8, "bf16", "bf16", t[8], 4096, 0)


@pytest.mark.parametrize("which", range(5))
def test_grad_norm(rr, which):
    t = [Stand(T if i == which else H, 4096 << i) for i in range(5)]
    refused(rr, rr.rr_grad_norm, t[:2], [8, 8], "bf16", 1.0, 1.0, t[2], t[3], t[4], 1 << 20, 0)


@pytest.mark.parametrize("which", range(12))
def test_adamw(rr, which):
    t = [Stand(T if i == which else H, 4096 << i) for i in range(15)]
    h = rr.rr_adamw_hyper(1e-3, 0.9, 0.99, 1e-8, 0.1, 1)
    if which < 11:
        refused(rr, rr.rr_adamw, t[0:2], t[2:4], t[4:6], t[6:8], t[8:10], [8, 8], "bf16", "bf16", h, t[10], 0)
    t = [Stand(T if i == which else H, 4096 << i) for i in range(15)]
    refused(rr, rr.rr_adamw8, t[0:2], t[2:4], t[4:6], t[6:8], t[8:10], t[10:12], t[12:14], [8, 8], "bf16", "bf16", h, 1,
            t[14], 0)


def test_addresses_and_empty_places_are_taken_as_they_are(rr):
    """Lists may mix tensors, addresses and None; only the tensors have a device."""
    h = rr.rr_adamw_hyper(1e-3, 0.9, 0.99, 1e-8, 0.1, 1)
    none = [None, None]
    rr.rr_adamw([Stand(H), None], none, none, none, None, [0, 0], "bf16", "bf16", h, None, 0)
    refused(rr, rr.rr_adamw, [None, Stand(T)], none, none, none, None, [0, 0], "bf16", "bf16", h, None, 0)
    rr.rr_adamw([4096, None], none, none, none, None, [0, 0], "bf16", "bf16", h, None, 0)
    with pytest.raises(ValueError, match="CUDA tensors"):
        rr.rr_adamw([Stand(-1), None], none, none, none, None, [0, 0], "bf16", "bf16", h, None, 0)


def test_cpu_tensors(rr, monkeypatch):
    """Refused as such, without a look at the current device, which may not exist."""
    from allgather_rr_allreduce_gb300 import _binding
    monkeypatch.setattr(_binding, "_device", lambda: pytest.fail("asked for the current device"))
    t = [Stand(-1, 4096 << i) for i in range(6)]
    with pytest.raises(ValueError, match="CUDA tensors"):
        rr.rr_layer_norm(*t, 1, 8, 8, 8, 1e-5, "bf16", "bf16", 0)
