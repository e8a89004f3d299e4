"""rr_grad_norm, rr_adamw and rr_adamw8 against plain implementations.

AdamW is compared in two ways.  Bit for bit with the formula evaluated
operation by operation in numpy's binary32 (the kernels fuse nothing, so every
state and weight has to agree exactly, whatever the alignment, the chunking
or the launch), and with the formula in 64 bits within a bound on the
roundings: e = 2^-24 a rounding of binary32, u the parameter type's.  A new
state is two products of rounded constants and one sum (5 e of the sum of
magnitudes; one product more for v), the step m / (sqrt(v) c + eps) adds five
roundings and the constants' three, and the weight two more.
"""
import math

import numpy as np
import pytest
import torch

from step_util import TINY, TORCH, U, U24, Guarded, generator, within

pytestmark = pytest.mark.gpu

BLOCK = 256
H = dict(lr=3e-3, beta1=0.9, beta2=0.97, eps=1e-8, weight_decay=0.1, step=3)


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.fail("this test needs a CUDA GPU")
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    return m


def hyper(rr, **kw):
    return rr.rr_adamw_hyper(*{**H, **kw}.values())


def host(t):
    """A CUDA tensor's values as float32 (exact for every type here)."""
    return t.float().cpu().numpy()


# ---------------------------------------------------------------- gradient norm
def norm_of(rr, tensors, dtype, inv_scale=1.0, max_norm=1.0, want=True):
    sizes = [t.numel() for t in tensors]
    n = rr.rr_grad_norm_workspace(len(sizes))
    ws, out = Guarded(n, torch.uint8), Guarded(2, torch.float32)
    rr.rr_grad_norm(tensors, sizes, dtype, inv_scale, max_norm, out.t[:1], out.t[1:], ws.t, n)
    norm, scale = out.t.tolist()
    ws.check("workspace")
    out.check("norm and scale")
    if want:
        exact = inv_scale * math.sqrt(sum(float(t.double().square().sum()) for t in tensors))
        check_norm(norm, scale, exact, inv_scale, max_norm, max([1] + sizes))
    return norm, scale


def check_norm(norm, scale, exact, inv_scale, max_norm, largest):
    """At most 64 products are added in sequence before a compensated sum takes
    over (binary64 above that): 70 e on the sum of squares, half of it on the
    norm, and a few roundings more."""
    assert abs(norm - exact) <= 40 * U24 * exact, (norm, exact)
    clip = inv_scale * min(1.0, max_norm / (exact + 1e-6))
    assert abs(scale - clip) <= 45 * U24 * clip, (scale, clip)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("sizes", [[1], [7], [0, 3, 0], [4096], [1000, 1, 70001, 3], [5] * 40, [300_001, 16_384],
                                   [3] * 1300, [2_000_003]])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_grad_norm(rr, dtype, sizes, shift):
    g = generator(len(sizes) + shift)
    tensors = []
    for n in sizes:
        flat = torch.randn(n + shift, generator=g, device="cuda").to(TORCH[dtype])
        tensors.append(flat[shift:])
    norm_of(rr, tensors, dtype)
    norm_of(rr, tensors, dtype, inv_scale=1 / 8, max_norm=1e9)
    norm_of(rr, tensors, dtype, max_norm=0.0)


def test_grad_norm_of_nothing(rr):
    for tensors in ([], [torch.empty(0, device="cuda")], [torch.zeros(1000, device="cuda")]):
        norm, scale = norm_of(rr, tensors, "fp32", inv_scale=0.5, want=False)
        assert norm == 0.0 and scale == 0.5


@pytest.mark.parametrize("value", [1e-30, 1e-42, 3e-16, 1e12, 2e13, 1e19, 3e38])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_grad_norm_far_from_one(rr, value, dtype):
    """Squares that leave binary32's range, alone and among ordinary values."""
    t = torch.full((10_001,), value, device="cuda").to(TORCH[dtype])
    if float(t[0]) == 0.0:
        pytest.skip("the value is zero in this type")
    exact = math.sqrt(float(t.double().square().sum()))
    norm, scale = norm_of(rr, [t], dtype, max_norm=float("inf"), want=False)
    if exact < 3.4e38:
        assert abs(norm - exact) <= max(45 * U24 * exact, 2.0 ** -149)
        assert scale == 1.0
    else:
        assert math.isinf(norm) and math.isnan(scale)
    t[::3] = 1.0
    exact = math.sqrt(float(t.double().square().sum()))
    norm, _ = norm_of(rr, [t], dtype, want=False)
    if exact < 3.4e38:
        assert abs(norm - exact) <= 45 * U24 * exact


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 5000, 10_000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_grad_norm_not_finite(rr, bad, at, dtype):
    t = torch.ones(10_001, device="cuda", dtype=TORCH[dtype])
    t[at] = bad
    norm, scale = norm_of(rr, [torch.ones(3, device="cuda", dtype=TORCH[dtype]), t], dtype, want=False)
    assert not math.isfinite(norm) and math.isnan(scale)
    assert math.isnan(norm) == math.isnan(bad)


def test_grad_norm_one_output_and_repeats(rr):
    t = torch.randn(1_000_001, generator=generator(4), device="cuda")
    n = rr.rr_grad_norm_workspace(1)
    ws = torch.empty(n, device="cuda", dtype=torch.uint8)
    a, b, s = (torch.zeros(1, device="cuda") for _ in range(3))
    rr.rr_grad_norm([t], [t.numel()], "fp32", 1.0, 1.0, a, None, ws, n)
    ws.fill_(255)
    rr.rr_grad_norm([t], [t.numel()], "fp32", 1.0, 1.0, None, s, ws, n)
    rr.rr_grad_norm([t], [t.numel()], "fp32", 1.0, 1.0, b, None, ws, n)
    assert torch.equal(a, b)
    check_norm(float(a), float(s), math.sqrt(float(t.double().square().sum())), 1.0, 1.0, t.numel())


def test_grad_norm_past_32_bit_offsets(rr):
    n = (1 << 32) + 12_345
    t = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    for at in (0, (1 << 31) + 1, (1 << 32) - 1, n - 1):
        t[at] = 3.0
    norm, _ = norm_of(rr, [t], "bf16", want=False)
    assert norm == 6.0


# ---------------------------------------------------------------- AdamW
def step_numpy(w, g, m, v, scale, h):
    """The formula operation by operation in binary32; returns weight, m, v, sqrt(v)."""
    f = np.float32
    g = g * f(scale)
    m = m * f(h["beta1"]) + g * f(1.0 - h["beta1"])
    v = v * f(h["beta2"]) + g * f(1.0 - h["beta2"]) * g
    r = np.sqrt(v)
    den = r * f(1.0 / math.sqrt(1.0 - h["beta2"] ** h["step"])) + f(h["eps"])
    w = w * f(1.0 - h["lr"] * h["weight_decay"]) - m / den * f(h["lr"] / (1.0 - h["beta1"] ** h["step"]))
    return w, m, v, r


def lists(sizes, shifts, seed, pd, gd, master):
    g = generator(seed)

    def make(dtype, scale, square=False):
        out = []
        for n, s in zip(sizes, shifts):
            b = Guarded(n, dtype, s)
            x = torch.randn(n, generator=g, device="cuda") * scale
            b.t.copy_(x.square() if square else x)
            out.append(b)
        return out

    L = {"p": make(TORCH[pd], 0.05), "g": make(TORCH[gd], 1e-2), "m": make(torch.float32, 3e-3),
         "v": make(torch.float32, 1e-2, True), "w": make(torch.float32, 0.05) if master else None}
    return L


def tensors(bufs):
    return None if bufs is None else [b.t for b in bufs]


def run_adamw(rr, L, sizes, pd, gd, scale=None, stream=None, **h):
    rr.rr_adamw(tensors(L["p"]), tensors(L["g"]), tensors(L["m"]), tensors(L["v"]), tensors(L["w"]), sizes, pd, gd,
                hyper(rr, **h), scale, stream)


def snapshot(L):
    return {k: None if b is None else [host(x.t) for x in b] for k, b in L.items()}


def check_adamw(L, old, pd, scale, h):
    for i in range(len(L["p"])):
        w0 = (old["w"] or old["p"])[i]
        with np.errstate(all="ignore"):
            w, m, v, _ = step_numpy(w0, old["g"][i], old["m"][i], old["v"][i], scale, h)
        assert np.array_equal(host(L["m"][i].t), m, equal_nan=True), f"tensor {i}: exp_avg"
        assert np.array_equal(host(L["v"][i].t), v, equal_nan=True), f"tensor {i}: exp_avg_sq"
        if L["w"]:
            assert np.array_equal(host(L["w"][i].t), w, equal_nan=True), f"tensor {i}: master"
        p = torch.from_numpy(w).to(TORCH[pd]).float().numpy()
        assert np.array_equal(host(L["p"][i].t), p, equal_nan=True), f"tensor {i}: param"
        assert np.array_equal(host(L["g"][i].t), old["g"][i], equal_nan=True), f"tensor {i}: grad was written"
    for bufs in L.values():
        for b in bufs or []:
            b.check()


TYPES = [("fp32", "fp32", False), ("bf16", "bf16", True), ("bf16", "bf16", False), ("bf16", "fp32", True),
         ("fp16", "fp16", True), ("fp16", "fp32", False), ("fp32", "bf16", False), ("fp32", "fp16", True)]
SIZES = [[1], [3, 4, 5], [0, 17, 0, 4096], [4097, 8191], [100_003], [33, 1] * 20, [7] * 450]


@pytest.mark.parametrize("pd,gd,master", TYPES)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_adamw_bit_for_bit(rr, pd, gd, master, sizes):
    """Aligned tensors, tensors off by the same number of elements (a shard
    inside flat buffers), and tensors off by different ones."""
    scale = torch.tensor([0.3], device="cuda")
    for shifts in ([0] * len(sizes), [i % 8 for i in range(len(sizes))], None):
        L = lists(sizes, shifts or [0] * len(sizes), len(sizes), pd, gd, master)
        if shifts is None:
            for k, name in enumerate(("p", "g", "m", "v")):
                L[name] = [shifted(b, (i + k) % 4) for i, b in enumerate(L[name])]
        old = snapshot(L)
        run_adamw(rr, L, sizes, pd, gd, scale)
        check_adamw(L, old, pd, float(scale), H)


def shifted(buf, shift):
    b = Guarded(buf.t.numel(), buf.t.dtype, shift)
    b.t.copy_(buf.t)
    return b


@pytest.mark.parametrize("pd,master", [("fp32", False), ("bf16", True)])
def test_adamw_against_64_bits(rr, pd, master):
    n = 50_001
    L = lists([n], [0], 77, pd, "fp32", master)
    d = {k: None if b is None else b[0].t.double() for k, b in L.items()}
    run_adamw(rr, L, [n], pd, "fp32")
    w0 = d["w"] if master else d["p"]
    b1, b2, t = H["beta1"], H["beta2"], H["step"]
    m = b1 * d["m"] + (1 - b1) * d["g"]
    v = b2 * d["v"] + (1 - b2) * d["g"] ** 2
    m_tol = 5 * U24 * ((b1 * d["m"]).abs() + ((1 - b1) * d["g"]).abs())
    v_tol = 6 * U24 * v
    move = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + H["eps"])
    w = w0 * (1 - H["lr"] * H["weight_decay"]) - H["lr"] * move
    w_tol = 4 * U24 * w0.abs() + H["lr"] * (14 * U24 * move.abs() + m_tol / m.abs().clamp(min=1e-30) * move.abs())
    within(L["m"][0].t, m, m_tol, "exp_avg")
    within(L["v"][0].t, v, v_tol, "exp_avg_sq")
    if master:
        within(L["w"][0].t, w, w_tol, "master")
    within(L["p"][0].t, w, w_tol * (1 + U[pd]) + U[pd] * w.abs() + TINY[pd], "param")


def test_adamw_no_scale_first_step_and_zero_betas(rr):
    for h in (dict(step=1), dict(beta1=0.0, beta2=0.0), dict(lr=0.0), dict(weight_decay=0.0, eps=0.0)):
        L = lists([1000], [0], 5, "fp32", "fp32", False)
        old = snapshot(L)
        run_adamw(rr, L, [1000], "fp32", "fp32", None, **h)
        check_adamw(L, old, "fp32", 1.0, {**H, **h})


@pytest.mark.parametrize("eight", [False, True])
def test_a_nan_scale_skips_the_step(rr, eight):
    nan = torch.tensor([float("nan")], device="cuda")
    sizes = [5000, 31, 3]
    if eight:
        L = lists8(sizes, [0, 1, 0], 6, "bf16", "fp32", True)
        old = snapshot8(L)
        run_adamw8(rr, L, sizes, "bf16", "fp32", nan)
        new = snapshot8(L)
    else:
        L = lists(sizes, [0, 1, 0], 6, "bf16", "fp32", True)
        old = snapshot(L)
        run_adamw(rr, L, sizes, "bf16", "fp32", nan)
        new = snapshot(L)
    for k in old:
        for a, b in zip(old[k] or [], new[k] or []):
            assert np.array_equal(a, b), k


def test_adamw_values_at_the_edge(rr):
    """Zero gradients and states, subnormals, infinities and NaN propagate as the formula says."""
    vals = [0.0, -0.0, 1e-45, 1e-38, 1e-20, 1e19, 3e38, float("inf"), -float("inf"), float("nan"), 1.0]
    n = len(vals) ** 2
    L = lists([n], [0], 8, "fp32", "fp32", False)
    g, m = np.meshgrid(np.float32(vals), np.float32(vals))
    L["g"][0].t.copy_(torch.from_numpy(g.reshape(-1).copy()))
    L["m"][0].t.copy_(torch.from_numpy(m.reshape(-1).copy()))
    L["v"][0].t[::2] = 0.0
    old = snapshot(L)
    run_adamw(rr, L, [n], "fp32", "fp32")
    check_adamw(L, old, "fp32", 1.0, H)


def test_adamw_on_a_stream_and_in_a_graph(rr):
    sizes = [20_000, 123]
    L = lists(sizes, [0, 2], 9, "bf16", "bf16", True)
    old = snapshot(L)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run_adamw(rr, L, sizes, "bf16", "bf16", None, side)
    for _ in range(2):
        graph.replay()
        check_adamw(L, old, "bf16", 1.0, H)
        old = snapshot(L)
    with torch.cuda.stream(side):
        run_adamw(rr, L, sizes, "bf16", "bf16")
    side.synchronize()
    check_adamw(L, old, "bf16", 1.0, H)


def test_pointer_arrays_made_before(rr):
    """Lists marshalled once, as a loop over the same tensors keeps them."""
    sizes = [3000, 17]
    L = lists(sizes, [0, 0], 10, "fp32", "fp32", False)
    old = snapshot(L)
    arrays = [rr.pointer_array(tensors(L[k])) for k in ("p", "g", "m", "v")]
    rr.rr_adamw(*arrays, None, sizes, "fp32", "fp32", hyper(rr))
    check_adamw(L, old, "fp32", 1.0, H)


def test_adamw_past_32_bit_offsets(rr):
    n = (1 << 31) + 5000
    p = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    at = [0, (1 << 31) - 4, n - 700]
    for a in at:
        for t in (p, g, m, v):
            t[a:a + 700].uniform_(0.5, 1.0, generator=generator(a + t.element_size()))
    keep = [[host(t[a:a + 700]) for t in (p, g, m, v)] for a in at]
    rr.rr_adamw([p], [g], [m], [v], None, [n], "bf16", "bf16", hyper(rr))
    for a, (p0, g0, m0, v0) in zip(at, keep):
        w, mw, vw, _ = step_numpy(p0, g0, m0, v0, 1.0, H)
        assert np.array_equal(host(m[a:a + 700]), mw) and np.array_equal(host(v[a:a + 700]), vw)
        assert np.array_equal(host(p[a:a + 700]), torch.from_numpy(w).bfloat16().float().numpy())
    for t in (p, g, m, v):
        assert int((t != 0).sum()) == 3 * 700


# ---------------------------------------------------------------- AdamW, 8-bit states
def code_values():
    """The 256 codes' values, from the format's definition."""
    out = np.zeros(256, np.float32)
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if e == 15 and f == 7 else -x if s else x
    return out


CODES = code_values()


def mix(x):
    x = (x ^ (x >> 16)) * 0x7FEB352D & 0xFFFFFFFF
    x = (x ^ (x >> 15)) * 0x68E31DA5 & 0xFFFFFFFF
    return x ^ (x >> 16)


def dither(n, tensor, seed):
    h = np.arange(n, dtype=np.uint64) * 0x9E3779B1 + mix((seed + (tensor + 1) * 0x9E3779B9) & 0xFFFFFFFF) & 0xFFFFFFFF
    h = (h ^ (h >> 16)) * 0x7FEB352D & 0xFFFFFFFF
    h = h ^ (h >> 15)
    return h & 0xFFFF, h >> 16


def encode(x, u, floor):
    """Codes and scales of binary32 values, in 64-bit arithmetic (exact but
    for the lift below 2^-6, which binary32 rounds)."""
    n = x.size
    blocks = -(-n // BLOCK)
    pad = np.zeros(blocks * BLOCK, np.float64)
    pad[:n] = x
    pad = pad.reshape(blocks, BLOCK)
    top = np.abs(pad).max(1)
    _, e = np.frexp(np.where(np.isfinite(top), top, 1.0))
    scale = np.ldexp(1.0, np.where(top == 0, -126, np.maximum(e - 8, -126)))  # a block of zeros: the least scale
    t = (np.abs(pad) / scale[:, None]).reshape(-1)[:n]
    if floor:
        t = np.where((t > 0) & (t < 2.0 ** -9), 2.0 ** -9, t)
    low = t < 2.0 ** -6
    t = np.where(low, np.float32(t).astype(np.float64), t)
    t = np.where(low, (np.float32(t) + np.float32(2.0 ** -6)).astype(np.float64), t)
    with np.errstate(all="ignore"):
        q = np.ldexp(1.0, np.frexp(t)[1] - 4)
        t = np.floor(t / q + (u + 0.5) / 65536) * q - np.where(low, 2.0 ** -6, 0.0)
    bad = ~np.isfinite(top)
    value = np.copysign(t, x)
    value[np.repeat(bad, BLOCK)[:n]] = 0.0
    return value.astype(np.float32), np.where(bad, np.nan, scale).astype(np.float32)


def lists8(sizes, shifts, seed, pd, gd, master, small=False):
    L = lists(sizes, shifts, seed, pd, gd, master)
    g = generator(seed + 1)
    blocks = [-(-n // BLOCK) for n in sizes]
    for name, high in (("m", 256), ("r", 128)):
        L[name], L[name + "s"] = [], []
        for n, k, s in zip(sizes, blocks, shifts):
            c = Guarded(n, torch.uint8, s)
            code = torch.randint(0, high, (n,), generator=g, device="cuda", dtype=torch.int32)
            code = torch.where(code % 128 == 127, code - 1, code)  # no NaN codes
            c.t.copy_(code)
            sc = Guarded(k, torch.float32, s % 2)
            sc.t.copy_(torch.exp2(torch.randint(-24, -18, (k,), generator=g, device="cuda").float()))
            L[name].append(c)
            L[name + "s"].append(sc)
    del L["v"]
    return L


def snapshot8(L):
    return {k: None if b is None else [x.t.cpu().numpy() if k in ("m", "r") else host(x.t) for x in b]
            for k, b in L.items()}


def run_adamw8(rr, L, sizes, pd, gd, scale=None, seed=12345, stream=None, **h):
    rr.rr_adamw8(tensors(L["p"]), tensors(L["g"]), tensors(L["m"]), tensors(L["ms"]), tensors(L["r"]),
                 tensors(L["rs"]), tensors(L["w"]), sizes, pd, gd, hyper(rr, **h), seed, scale, stream)


def decoded(code, scale, n):
    return CODES[code] * np.repeat(scale, BLOCK)[:n]


def check_adamw8(L, old, sizes, pd, scale, seed, h):
    for i, n in enumerate(sizes):
        if n == 0:
            continue
        with np.errstate(all="ignore"):
            m0 = decoded(old["m"][i], old["ms"][i], n)
            r0 = decoded(old["r"][i], old["rs"][i], n)
            w, m, v, r = step_numpy((old["w"] or old["p"])[i], old["g"][i], m0, r0 * r0, scale, h)
        if L["w"]:
            assert np.array_equal(host(L["w"][i].t), w, equal_nan=True), f"tensor {i}: master"
        assert np.array_equal(host(L["p"][i].t), torch.from_numpy(w).to(TORCH[pd]).float().numpy(), equal_nan=True), i
        low, high = dither(n, i, seed)
        for name, x, u, floor in (("m", m, low, False), ("r", r, high, True)):
            value, sc = encode(x, u, floor)
            assert np.array_equal(host(L[name + "s"][i].t), sc, equal_nan=True), f"tensor {i}: scale of {name}"
            got = CODES[L[name][i].t.cpu().numpy()]
            assert np.array_equal(got, value), f"tensor {i}: codes of {name}"
    for bufs in L.values():
        for b in bufs or []:
            b.check()


@pytest.mark.parametrize("pd,gd,master", TYPES)
@pytest.mark.parametrize("sizes", [[1], [255, 256, 257], [0, 17, 0, 4096], [9_999], [300, 1] * 20, [7] * 450],
                         ids=lambda s: f"{len(s)}x{max(s)}")
def test_adamw8_bit_for_bit(rr, pd, gd, master, sizes):
    scale = torch.tensor([0.3], device="cuda")
    for shifts in ([0] * len(sizes), [i % 5 for i in range(len(sizes))]):
        L = lists8(sizes, shifts, len(sizes), pd, gd, master)
        old = snapshot8(L)
        run_adamw8(rr, L, sizes, pd, gd, scale)
        check_adamw8(L, old, sizes, pd, float(scale), 12345, H)


def test_adamw8_from_zero_states_and_large_seed(rr):
    sizes = [1000, 300]
    L = lists8(sizes, [0, 0], 3, "fp32", "fp32", False)
    for name in ("m", "ms", "r", "rs"):
        for b in L[name]:
            b.t.zero_()
    L["g"][0].t[:256] = 0.0      # a block of zeros keeps zeros
    L["g"][1].t[5] = 0.0
    for k in range(3):
        old = snapshot8(L)
        run_adamw8(rr, L, sizes, "fp32", "fp32", None, 0xFFFFFFF0 + k, step=k + 1)
        check_adamw8(L, old, sizes, "fp32", 1.0, 0xFFFFFFF0 + k, {**H, "step": k + 1})
    assert int(L["m"][0].t[:256].sum()) == 0 and int(L["r"][0].t[:256].sum()) == 0


@pytest.mark.parametrize("size", [1e-44, 1e-37, 1e-30, 1e-19, 1e-12, 1e10, 1e18, 3e38])
def test_adamw8_magnitudes(rr, size):
    """Scales from the smallest to the largest, where squares of gradients vanish or overflow."""
    n = 700
    L = lists8([n], [0], 4, "fp32", "fp32", False)
    for name in ("m", "ms", "r", "rs"):
        L[name][0].t.zero_()
    L["g"][0].t.copy_((torch.rand(n, device="cuda", generator=generator(1)) * 2 - 1) * size)
    old = snapshot8(L)
    run_adamw8(rr, L, [n], "fp32", "fp32")
    check_adamw8(L, old, [n], "fp32", 1.0, 12345, H)


def test_adamw8_not_finite_values_spoil_their_block_only(rr):
    n = 1024
    L = lists8([n], [0], 14, "fp32", "fp32", False)
    L["g"][0].t[300] = float("nan")
    L["g"][0].t[600] = float("inf")
    old = snapshot8(L)
    run_adamw8(rr, L, [n], "fp32", "fp32")
    check_adamw8(L, old, [n], "fp32", 1.0, 12345, H)
    assert np.isnan(host(L["ms"][0].t)).tolist() == [False, True, True, False]
    assert np.isnan(host(L["p"][0].t)).nonzero()[0].tolist() == [300, 600]


def test_adamw8_rounding_is_unbiased(rr):
    """Over S seeds the mean of the stored value is the unrounded one: each
    rounding is off by less than one grid step q with a standard deviation of
    at most q / 2, so the mean is within 6 * q / (2 sqrt(S)) (and 2^-17 q of
    the dither's own grain).  1000 values at 6 standard deviations: a false
    alarm has probability below 1e-5."""
    n, S = 1024, 400
    L = lists8([n], [0], 15, "fp32", "fp32", False)
    old = {k: None if b is None else b[0].t.clone() for k, b in L.items()}
    before = snapshot8(L)
    _, m, v, r = step_numpy(before["p"][0], before["g"][0], decoded(before["m"][0], before["ms"][0], n),
                            decoded(before["r"][0], before["rs"][0], n) ** 2, 1.0, H)
    total = {"m": np.zeros(n), "r": np.zeros(n)}
    for k in range(S):
        for name, b in L.items():
            if b is not None:
                b[0].t.copy_(old[name])
        run_adamw8(rr, L, [n], "fp32", "fp32", None, 1000 + k)
        for name in total:
            total[name] += decoded(L[name][0].t.cpu().numpy(), host(L[name + "s"][0].t), n)
    for name, x in (("m", m), ("r", r)):
        sc = np.repeat(host(L[name + "s"][0].t), BLOCK)[:n]
        t = np.abs(x) / sc
        q = np.ldexp(1.0, np.maximum(np.frexp(t)[1], -5) - 4) * sc
        x = np.where((name == "r") & (t < 2.0 ** -9), 2.0 ** -9 * sc, x)
        off = np.abs(total[name] / S - x) / q
        assert off.max() <= 6 / (2 * math.sqrt(S)) + 2.0 ** -16, (name, off.max())


def test_adamw8_slow_averages_move(rr):
    """With beta2 = 0.999 and no gradient, sqrt(v) shrinks by 0.05 % a step, a
    hundredth of the codes' spacing: rounding to nearest would never move it.
    After 400 steps it should be 0.999^200 = 0.8187 of itself: the mean over
    n values, each a walk of 400 roundings of at most q / 2 = 1/16 relative
    deviation, is within 6 * sqrt(400) / 16 / sqrt(n) of it."""
    n, steps = 1 << 16, 400
    L = lists8([n], [0], 16, "fp32", "fp32", False)
    L["g"][0].t.zero_()
    L["m"][0].t.zero_()
    L["r"][0].t.fill_(0x70)      # 128
    L["rs"][0].t.fill_(2.0 ** -20)
    for k in range(steps):
        run_adamw8(rr, L, [n], "fp32", "fp32", None, k, beta2=0.999, step=1000 + k)
    r = decoded(L["r"][0].t.cpu().numpy(), host(L["rs"][0].t), n).astype(np.float64) / (128 * 2.0 ** -20)
    assert abs(r.mean() - 0.999 ** (steps / 2)) <= 6 * math.sqrt(steps) / 16 / math.sqrt(n), r.mean()


def test_adamw8_past_32_bit_offsets(rr):
    n = (1 << 32) + 3 * BLOCK + 77
    p = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    m, r = (torch.zeros(n, device="cuda", dtype=torch.uint8) for _ in range(2))
    ms, rs = (torch.zeros(-(-n // BLOCK), device="cuda") for _ in range(2))
    at = [0, 1 << 31, (1 << 32) - BLOCK, (1 << 32) + 3 * BLOCK]
    for a in at:
        for t in (p, g):
            t[a:a + BLOCK].uniform_(0.5, 1.0, generator=generator(a + 1))
    keep = [[host(t[a:a + BLOCK]) for t in (p, g)] for a in at]
    rr.rr_adamw8([p], [g], [m], [ms], [r], [rs], None, [n], "bf16", "bf16", hyper(rr), 5)
    low, high = dither(BLOCK * 4, 0, 5)   # the element's index enters modulo 2^32
    for a, (p0, g0) in zip(at, keep):
        w, mw, vw, rw = step_numpy(p0, g0, 0 * g0, 0 * g0, 1.0, H)
        assert np.array_equal(host(p[a:a + BLOCK]), torch.from_numpy(w).bfloat16().float().numpy())
        b = a // BLOCK
        got = CODES[m[a:a + BLOCK].cpu().numpy()] * float(ms[b])
        assert np.abs(got / mw - 1).max() <= 1 / 8
        if a in (0, (1 << 32) + 3 * BLOCK):
            k = a % (1 << 32)
            value, sc = encode(mw, low[k:k + len(p0)], False)
            assert float(ms[b]) == sc[0] and np.array_equal(CODES[m[a:a + BLOCK].cpu().numpy()], value)
            value, sc = encode(rw, high[k:k + len(p0)], True)
            assert float(rs[b]) == sc[0] and np.array_equal(CODES[r[a:a + BLOCK].cpu().numpy()], value)
    assert int((p != 0).sum()) == sum(len(k[0]) for k in keep)
