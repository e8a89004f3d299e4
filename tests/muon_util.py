"""Newton-Schulz products in 64 bits, and a model of what the kernels' arithmetic
may leave in them.

The model: an operand is a pair of binary16 pieces, off by 2^-22 of its value and
2^-36 at least (half the smallest binary16 subnormal over the scale 2^11); a
product drops lo lo (2^-22 of the terms' magnitudes) and sums at most 8
instructions at a time in an accumulator that loses up to 2^-24 of the running sum
at each (8 * 2^-24 = 2^-21), the rest rounding to nearest.  So each product is off
by at most 2^-22 + 2^-21 < 2^-20 of |X| |Y|.  The iteration amplifies that; by how
much is seen from 64-bit runs whose operands and products are perturbed at random
within those bounds, and a result may be three times as far off as such a run."""
import torch

COEFS = [(3.4445, -4.7750, 2.0315)] * 5


def products(x, coefs, eps=1e-7, noise=None):
    """noise: a generator; perturbs each step's operands and products within the model's bounds."""
    tall = x.shape[0] > x.shape[1]
    x = x.double()
    x = x.t() if tall else x
    x = x / (torch.linalg.matrix_norm(x) + eps) if noise is None else x / (torch.linalg.matrix_norm(x) + eps) * (1 + 2.0 ** -23)

    def rough(v):
        if noise is None:
            return v
        r = torch.rand(v.shape, generator=noise, device=v.device, dtype=torch.float64) * 2 - 1
        return v + r * torch.clamp(v.abs() * 2.0 ** -22, min=2.0 ** -36)

    def mul(p, q):
        d = p @ q
        if noise is None:
            return d
        r = torch.rand(d.shape, generator=noise, device=d.device, dtype=torch.float64) * 2 - 1
        return d + r * 2.0 ** -20 * (p.abs() @ q.abs())

    x = rough(x)
    for a, b, c in coefs:
        m = rough(mul(x, x.t()))
        p = c * mul(m, m) + b * m
        p.diagonal().add_(a)
        x = mul(rough(p), x)
        x = rough(x)
    return x.t() if tall else x


def allowed(x, coefs, eps=1e-7, seed=0):
    """Exact result and the relative 2-norm that the model allows."""
    want = products(x, coefs, eps)
    g = torch.Generator(device=x.device)
    off = 0.0
    for k in range(2):
        g.manual_seed(seed + k)
        off = max(off, float((products(x, coefs, eps, g) - want).norm()))
    return want, 3 * off / max(float(want.norm()), 1e-300)


def near(got, want, tol, unit, what=""):
    """Relative 2-norm within tol and the type's rounding, single values within ten times that of the size of the rows' mean."""
    got = got.double()
    n = float(want.norm())
    off = float((got - want).norm())
    assert off <= (tol + unit) * n, f"{what}: off by {off / n:.3g}, {tol + unit:.3g} allowed"
    rms = n / want.numel() ** 0.5
    worst = float(((got - want).abs() / torch.clamp(want.abs(), min=rms)).max())
    assert worst <= 10 * (tol + unit), f"{what}: a value is off by {worst:.3g}, {10 * (tol + unit):.3g} allowed"
