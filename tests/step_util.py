"""Helpers of the training-step operators' tests: buffers between canaries at
a chosen alignment, and units of rounding."""
import torch

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}   # relative rounding to the type
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}  # half its smallest subnormal
U24 = 2.0 ** -24

GUARD = 64   # canary bytes on each side
CANARY = 0xA5


class Guarded:
    """A flat tensor of n elements `shift` elements past a 16-byte boundary,
    with canary bytes before and after it."""

    def __init__(self, n, dtype, shift=0, device="cuda"):
        eb = torch.empty((), dtype=dtype).element_size()
        self.lead = GUARD + shift * eb
        self.bytes = n * eb
        self.raw = torch.full((self.lead + self.bytes + GUARD + 16,), CANARY, dtype=torch.uint8, device=device)
        # a byte view at any element offset: reinterpret through the address-aligned slice
        self.t = self.raw[self.lead:self.lead + self.bytes].view(dtype)

    def check(self, what=""):
        head, tail = self.raw[:self.lead], self.raw[self.lead + self.bytes:]
        assert bool((head == CANARY).all()) and bool((tail == CANARY).all()), f"{what}: canary overwritten"


def guarded_like(values, dtype, shift=0):
    g = Guarded(values.numel(), dtype, shift)
    g.t.copy_(values.reshape(-1).to(dtype))
    return g


def generator(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def within(got, want, tol, what=""):
    """Every element of got within tol (a tensor) of want (float64); NaN and
    infinities of want must match."""
    got, tol = got.double(), torch.broadcast_to(tol, want.shape)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert bool((torch.isnan(got) == torch.isnan(want)).all()), f"{what}: NaN in other places"
    assert bool((got[~fine & ~torch.isnan(want)] == want[~fine & ~torch.isnan(want)]).all()), f"{what}: infinities"
    off = (got - want).abs()[fine]
    room = tol[fine]
    bad = off > room
    if bool(bad.any()):
        i = int((off / room.clamp(min=1e-300)).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; worst {float(off[i])} "
                             f"where {float(room[i])} is allowed")
