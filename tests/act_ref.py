"""The activation operators' definitions in 64 bits, and how far an fp32
evaluation in the kernels' order may be from them.

Error bounds count roundings.  U = 2^-24 is the most one fp32 operation is off
relative to its result, HALF[dtype] the most one rounding to an output type
is, and a sum of n terms in which no term passes through more than d additions
is off by at most d U times the sum of magnitudes.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: torch.finfo(torch.float32).eps / 2, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
TINY = 4e-36        # results whose exponential under- or overflows: e^-88 times the largest inputs of the tests


def depth(cols):
    """Most additions a term of a row's sum passes through: 8 in a chunk, the
    chunks of a thread (2, or one per 8192 columns of a wide row), 6 in the
    wave, 16 waves, and the division by cols."""
    return 8 + max(2, -(-cols // 8192)) + 6 + 16 + 1


def stats(s, eps, layer):
    """mean, rstd of the rows of s (float64)."""
    mu = s.mean(1) if layer else torch.zeros(s.shape[0], dtype=torch.float64)
    return mu, ((s - mu[:, None]).square().mean(1) + eps).rsqrt()


def norm(s, w, b, eps, layer):
    """y, mean, rstd and the bounds on their errors in fp32."""
    d = depth(s.shape[1])
    mu, r = stats(s, eps, layer)
    mu_err = d * U * s.abs().mean(1) if layer else torch.zeros_like(mu)
    # the variance is of c = s - mu': the mean's own error e shifts every c by
    # e, which changes the mean square by 2 e mean(c) + e^2 <= e^2 + rounding,
    # and c^2 carries three roundings; 1 / sqrt halves that and adds three
    var = (s - mu[:, None]).square().mean(1)
    var_err = (d + 3) * U * var + mu_err ** 2 + 2 * mu_err * var.sqrt() * U * d
    r_err = r * (0.5 * var_err / (var + eps).clamp(min=1e-300) + 4 * U)
    c = (s - mu[:, None]) * r[:, None] * w
    y = c + b
    err = (c.abs() * (r_err / r)[:, None] + mu_err[:, None] * r[:, None] * w.abs() + 4 * U * c.abs() + 2 * U * y.abs())
    return y, err, mu, mu_err, r, r_err


def norm_grad(dy, s, mu, r, w, dsum, layer, per_part):
    """dx, dweight, dbias and bounds; mu and r are inputs (exact), per_part
    the most additions of a column sum's terms."""
    d, mu, r = depth(s.shape[1]), mu[:, None], r[:, None]
    h, g = (s - mu) * r, dy * w
    mgh = (g * h).mean(1, keepdim=True)
    mg = g.mean(1, keepdim=True) if layer else torch.zeros_like(mgh)
    dx = r * (g - mg - h * mgh) + dsum
    mgh_err = (d + 5) * U * (g * h).abs().mean(1, keepdim=True)
    mg_err = (d + 2) * U * g.abs().mean(1, keepdim=True) if layer else 0.0
    err = r * (4 * U * g.abs() + mg_err + 3 * U * mg.abs() + h.abs() * (mgh_err + 6 * U * mgh.abs())) + 2 * U * dx.abs() \
        + U * dsum.abs()
    dw, db = (dy * h).sum(0), dy.sum(0)
    return dx, err, dw, (per_part + 4) * U * (dy * h).abs().sum(0), db, per_part * U * dy.abs().sum(0)


def gate(x, act):
    """act(x), act'(x) in float64 and bounds on their fp32 errors."""
    if act == "gelu":
        p, phi = 0.5 * torch.erfc(-x * math.sqrt(0.5)), torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        a, d = x * p, p + x * phi
        # an argument of erfc off by 2 U relative shifts P by 2 U |x| phi(x)
        # (2 x^2 U P in the lower tail; 3 U for the shift's own growth there);
        # 4 ulp for erfc itself.  The density's exponent carries four roundings.
        p_err = 3 * U * x.abs() * phi + 10 * U * p
        d_err = p_err + x.abs() * phi * (2 * x * x + 8) * U + 2 * U * d.abs()
        return a, d, x.abs() * p_err + 2 * U * a.abs() + TINY, d_err + TINY
    if act == "silu":
        z, slope, k = x, torch.ones_like(x), 2
    else:
        z = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
        slope, k = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x), 4
    # e^-z from a product with k roundings: k |z| U, 2 U for the exponential, 3 for 1 / (1 + .), 1 for x s
    s, t = torch.special.expit(z), torch.special.expit(-z)
    a = x * s
    d = s + a * t * slope
    rel = (k * z.abs() + 8) * U
    err = rel * (s + a.abs() * t * slope + a.abs() * s * slope) + U * a.abs() * slope + 8 * U * a.abs() * t * slope
    return a, d, a.abs() * rel + TINY, err + 2 * U * d.abs() + TINY


def within(got, want, err, what, dtype=None):
    """|got - want| <= err plus the output type's rounding, NaN where NaN."""
    dtype = got.dtype if dtype is None else dtype
    got, want = got.detach().cpu().double(), want.cpu()
    tol = err * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + 1e-37
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    # an infinite result has an infinite or undefined bound
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    bad = ((got - want).abs() > tol) & ~torch.isnan(want) & ~inf
    if bool(bad.any()):
        k = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} values off, first at {k}: got {got[k]!r} want {want[k]!r} "
                             f"tolerance {tol[k]!r}")
