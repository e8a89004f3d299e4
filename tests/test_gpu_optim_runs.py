"""Lists long enough that blocks and warps of the gradient norm and the AdamW
steps work through many pieces of their own: rings used again and again, runs of
blocks that begin and end inside tensors, stretches that cross from one tensor to
the next, short last blocks in the middle of a list.  Bit for bit and bounds as in
test_gpu_adamw.py."""
import pytest
import torch

from step_util import TORCH, generator
from test_gpu_adamw import (H, TYPES, check_adamw, check_adamw8, lists, lists8, norm_of, rr, run_adamw,  # noqa: F401
                            run_adamw8, shifted, snapshot, snapshot8)

pytestmark = pytest.mark.gpu

SCALE = 0.3
# about 20 blocks of 256 to a warp where one thread block has an SM
SIZES8 = [1_000_003, 77, 2_500_100, 256 * 40 + 3, 5, 256 * 700, 300_001, 0, 2_200_011, 255, 400_000]


@pytest.mark.parametrize("pd,gd,master", TYPES)
@pytest.mark.parametrize("shifts", [[0] * len(SIZES8), [0, 1, 0, 3, 0, 0, 1, 0, 1, 0, 0]], ids=["aligned", "mixed"])
def test_adamw8_many_blocks_to_a_warp(rr, pd, gd, master, shifts):  # noqa: F811
    scale = torch.tensor([SCALE], device="cuda")
    L = lists8(SIZES8, shifts, 40, pd, gd, master)
    old = snapshot8(L)
    run_adamw8(rr, L, SIZES8, pd, gd, scale)
    check_adamw8(L, old, SIZES8, pd, float(scale), 12345, H)


def test_adamw8_more_than_a_run_to_a_warp(rr):  # noqa: F811
    """16-bit weights, where more thread blocks share an SM and a warp has fewer blocks."""
    sizes = [17_000_001, 300, 3_000_000]
    L = lists8(sizes, [0, 0, 0], 41, "bf16", "bf16", False)
    old = snapshot8(L)
    run_adamw8(rr, L, sizes, "bf16", "bf16")
    check_adamw8(L, old, sizes, "bf16", 1.0, 12345, H)


@pytest.mark.parametrize("pd,gd,master", TYPES)
@pytest.mark.parametrize("how", ["aligned", "alike", "each its own"])
def test_adamw_many_chunks_to_a_block(rr, pd, gd, master, how):  # noqa: F811
    sizes = [3_000_001, 17, 2_500_000, 4096, 1_000_003]
    scale = torch.tensor([SCALE], device="cuda")
    L = lists(sizes, [1, 2, 3, 0, 2] if how == "alike" else [0] * 5, 42, pd, gd, master)
    if how == "each its own":
        for k, name in enumerate(("p", "g", "m", "v")):
            L[name] = [shifted(b, (i + k) % 4) for i, b in enumerate(L[name])]
    old = snapshot(L)
    run_adamw(rr, L, sizes, pd, gd, scale)
    check_adamw(L, old, pd, float(scale), H)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("sizes", [[40_000_001], [9_000_001, 3, 16_000_000, 0, 7_777_777] + [100_003] * 60])
@pytest.mark.parametrize("shift", [0, 1])
def test_grad_norm_many_chunks_to_a_block(rr, dtype, sizes, shift):  # noqa: F811
    g = generator(len(sizes) + shift)
    tensors = [torch.randn(n + shift, generator=g, device="cuda").to(TORCH[dtype])[shift:] for n in sizes]
    norm_of(rr, tensors, dtype)
    tensors[0].copy_(1.1)   # alike throughout, so that roundings add up
    norm_of(rr, tensors, dtype, inv_scale=1 / 8, max_norm=1e9)
