"""Plain 64-bit forms of the transformer-block operators and the error bounds
that the tests of the HIP path hold it to.

The bounds count roundings (u = 2^-24 each): a row's sum passes at most 24
additions (three within a 16-byte group, four groups, ten lane steps, and the
joins of waves), the FP32 activations are good to a few units, a product has
the a-priori bound of the GEMM's own tests.  They are written per element,
from the magnitudes of the terms that are added.
"""
import math

import torch

U = 2.0**-24
ACTS = ("identity", "relu", "silu", "gelu", "gelu_tanh", "tanh")
DELTA = {"NATIVE_F32": 0.0, "BF16X9": 0.0, "AUTO": 0.0, "BF16X6": 2.0**-22, "BF16X3": 2.0**-14, "BF16X1": 2.0**-7}
C = math.sqrt(2.0 / math.pi)
A3 = 0.044715


def f64(t):
    return None if t is None else t.detach().double()


def act(name, z):
    if name == "identity":
        return z
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * C * (z + A3 * z**3))
    return torch.tanh(z)


def slopes(name, z):
    """act', act'' and the magnitudes of the terms they are made of."""
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    if name == "identity":
        return one, zero, one, zero
    if name == "relu":
        return (z > 0).double(), zero, one, zero
    if name == "gelu":
        pdf = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        cdf = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        # (the exponent -z^2 / 2 carries its own rounding)
        return (cdf + z * pdf, pdf * (2 - z * z), cdf + z.abs() * pdf * (1 + z * z), pdf * (2 + z * z) * (1 + z * z))
    if name == "tanh":
        s = 4 * torch.sigmoid(2 * z) * torch.sigmoid(-2 * z)
        return s, -2 * torch.tanh(z) * s, s, 2 * s
    p, p1, p2 = (z, one, zero) if name == "silu" else (2 * C * (z + A3 * z**3), 2 * C * (1 + 3 * A3 * z * z), 12 * C * A3 * z)
    s, t = torch.sigmoid(p), torch.sigmoid(-p)
    d1, d2 = s + z * s * t * p1, s * t * (2 * p1 + z * (p2 + (t - s) * p1 * p1))
    # p's rounding moves s by s t |p|
    return (d1, d2, (s + z.abs() * s * t * p1.abs()) * (1 + t * p.abs() + s * t * p.abs()),
            s * t * (2 * p1.abs() + z.abs() * (p2.abs() + p1 * p1)) * (1 + p.abs()))


def act_bound(name, z):
    """Error of act(z) itself.  FP32 reciprocals and exponentials below the
    smallest normal number, 2^-126, are zero: a sigmoid is, from z = -87.4 on
    (its exponential overflows at 88.8), which takes up to 88.8 * 2^-126 <
    2^-119 from z * sigmoid(z)."""
    v = act(name, z).abs()
    if name in ("identity", "relu"):
        return torch.zeros_like(v)
    if name == "gelu_tanh":
        p = 2 * C * (z + A3 * z**3)
        return 16 * U * v * (1 + p.abs() * torch.sigmoid(-p)) + 2.0**-119
    if name == "gelu":
        return 16 * U * v * (1 + z * z) + 2.0**-119
    return 16 * U * v + 2.0**-119


def worst(got, ref, bound):
    """max |got - ref| / bound; infinite where only one of them is finite."""
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), "non-finite result"
    if got.numel() == 0:
        return 0.0
    d = (got.double() - ref).abs()
    return float(torch.where(d == 0, torch.zeros_like(d), d / bound).max())


# ---- layer norm ---------------------------------------------------------------------

def norm_parts(x, eps):
    x = f64(x)
    mu = x.mean(-1, keepdim=True)
    r = torch.rsqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    return (x - mu) * r, r, x.abs().mean(-1, keepdim=True) * r


def norm(x, w, b, eps):
    xhat, r, mx = norm_parts(x, eps)
    w = torch.ones_like(xhat[:1]) if w is None else f64(w)
    b = torch.zeros_like(xhat[:1]) if b is None else f64(b)
    y = xhat * w + b
    return y, w.abs() * (24 * U * mx + 32 * U * xhat.abs()) + 4 * U * (y.abs() + b.abs())


def norm_backward(x, w, dy, eps):
    xhat, r, mx = norm_parts(x, eps)
    dy = f64(dy)
    a = dy if w is None else dy * f64(w)
    m = lambda t: t.mean(-1, keepdim=True)
    dx = r * (a - m(a) - xhat * m(a * xhat))
    size = r * (a.abs() + m(a.abs()) + xhat.abs() * m((a * xhat).abs())
                + mx * (m((a * xhat).abs()) + xhat.abs() * m(a.abs())))
    rows = x.shape[0]
    sums = (dy.abs() * (xhat.abs() + mx)).sum(0)
    # (a workgroup's threads add at most rows / 8 + 8 rows each one after the
    # other, the joins add 24 more)
    depth = 96 + min(rows, 64 + rows / 8)
    return (dx, 192 * U * size), ((dy * xhat).sum(0), depth * U * sums), (dy.sum(0), depth * U * dy.abs().sum(0))


def norm_backward2(x, w, dy, v, p, q, eps):
    xhat, r, mx = norm_parts(x, eps)
    dy = f64(dy)
    zero = torch.zeros_like(xhat)
    w = torch.ones_like(xhat[:1]) if w is None else f64(w)
    v = zero if v is None else f64(v)
    p = zero[:1] if p is None else f64(p)
    q = zero[:1] if q is None else f64(q)
    a = dy * w
    m = lambda t: t.mean(-1, keepdim=True)
    s = r * (v - m(v) - xhat * m(v * xhat))
    ss = r * (v.abs() + m(v.abs()) + xhat.abs() * m((v * xhat).abs()))
    gdy = w * s + p * xhat + q
    pa = a - m(a) - xhat * m(a * xhat)
    pas = a.abs() + m(a.abs()) + xhat.abs() * m((a * xhat).abs())
    h = p * dy - r * (a * m(v * xhat) + v * m(a * xhat))
    hs = (p * dy).abs() + r * (a.abs() * m((v * xhat).abs()) + v.abs() * m((a * xhat).abs()))
    gx = r * (h - m(h) - xhat * m(h * xhat)) - xhat * r * r * m(v * pa)
    gxs = r * (hs + m(hs) + xhat.abs() * m(hs * xhat.abs())) + xhat.abs() * r * r * m(v.abs() * pas)
    gw = (dy * s).sum(0)
    k = 1 + mx
    depth = 320 + min(x.shape[0], 64 + x.shape[0] / 8)
    return ((gdy, 320 * U * k * (w.abs() * ss + (p * xhat).abs() + p.abs() * mx + q.abs())),
            (gx, 320 * U * k * (gxs + xhat.abs() * m(hs) + xhat.abs() * r * m(v.abs() * pas))),
            (gw, depth * U * ((dy.abs() * ss * k).sum(0))))


# ---- products --------------------------------------------------------------------------

def product(a, w, bias, mode):
    """(z, bound) of a w^T + bias for 64-bit a, w."""
    z = a @ w.t()
    size = a.abs() @ w.abs().t()
    b = 0.0 if bias is None else f64(bias)
    z = z + b
    K = a.shape[1]
    return z, ((2 * K + 10) * U + DELTA[mode]) * size + 2 * U * (z.abs() + size)
