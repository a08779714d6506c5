"""The attention operators' definitions in 64 bits, with a bound on what FP32
arithmetic of the same formulas may be off.

``Bounded`` carries a value and a bound of its error through each operation
(running error analysis): an FP32 operation adds u = 2^-24 of its result's
size, a sum of n numbers in any order n u of the sum of their absolute values,
on top of what its operands bring.  A matrix product of n terms adds (2 n + 10)
u of the sum of |a b|: 2 u an addition on the matrix unit, as for the GEMMs
(tests/gpu_helpers.py); split operands leave out 2^-25 of |a b|, and their six
products' additions, 6 / 32 n instructions, are fewer than 2 n.  The bound is
first order, times 1.01 for the rest.
"""
import math

import torch

U = 2.0 ** -24


class Bounded:
    def __init__(self, v, e=None):
        self.v = v
        self.e = torch.zeros_like(v) if e is None else e

    def rounded(self, n=1.0):
        return Bounded(self.v, self.e + n * U * self.v.abs())

    def __add__(self, o):
        return Bounded(self.v + o.v, self.e + o.e).rounded()

    def __sub__(self, o):
        return Bounded(self.v - o.v, self.e + o.e).rounded()

    def __mul__(self, o):
        if not isinstance(o, Bounded):
            return Bounded(self.v * o, self.e * abs(o)).rounded(2.0)   # (the constant's rounding too)
        return Bounded(self.v * o.v, self.e * o.v.abs() + o.e * self.v.abs()).rounded()

    def __matmul__(self, o):
        a, b = self.v.abs(), o.v.abs()
        n = 2 * self.v.shape[-1] + 10
        return Bounded(self.v @ o.v, self.e @ b + a @ o.e + n * U * (a @ b))

    def sum(self, dim, keepdim=False, extra=0):
        n = self.v.shape[dim] + 2 + extra
        return Bounded(self.v.sum(dim, keepdim=keepdim),
                       self.e.sum(dim, keepdim=keepdim) + n * U * self.v.abs().sum(dim, keepdim=keepdim))

    @property
    def T(self):
        return Bounded(self.v.transpose(-1, -2), self.e.transpose(-1, -2))

    def where(self, cond):
        zero = torch.zeros((), dtype=self.v.dtype, device=self.v.device)
        return Bounded(torch.where(cond, self.v, zero), torch.where(cond, self.e, zero))


def _rows(t, share):
    """[batch, tokens, heads, dim] to [batch, heads, tokens, dim], heads repeated `share` times."""
    return Bounded(t.double().transpose(1, 2).repeat_interleave(share, dim=1).contiguous())


def _back(b):
    return Bounded(b.v.transpose(1, 2), b.e.transpose(1, 2))


def _shared(b, share):
    """The sum over the heads that share a key head."""
    n, h, t, d = b.v.shape
    return _back(Bounded(b.v.reshape(n, h // share, share, t, d), b.e.reshape(n, h // share, share, t, d)).sum(2))


def alive_keys(k, bias=None, mask=None, lengths=None):
    batch, keys = k.shape[:2]
    alive = torch.ones(batch, keys, dtype=torch.bool, device=k.device)
    if lengths is not None:
        alive &= torch.arange(keys, device=k.device) < lengths[:, None]
    if mask is not None:
        alive &= mask
    if bias is not None:
        alive &= bias != -math.inf
    return alive


class Attention:
    """The forward pass, its gradients and theirs, by the formulas of include/emu_attention.h."""

    def __init__(self, q, k, v, bias=None, mask=None, lengths=None, scale=None):
        self.scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
        self.share = q.shape[2] // k.shape[2]
        alive = alive_keys(k, bias, mask, lengths)
        self.alive = alive[:, None, None, :]
        dead = ~alive[:, :, None, None]
        self.dead = dead
        self.q = _rows(q, 1)
        self.k, self.v = (_rows(t.masked_fill(dead, 0.0), self.share) for t in (k, v))
        t = (self.q @ self.k.T) * self.scale
        if bias is not None:
            t = t + Bounded(bias.double().masked_fill(~alive, 0.0)[:, None, None, :])
        t = Bounded(t.v.masked_fill(~self.alive, -math.inf), t.e.masked_fill(~self.alive, 0.0))
        if t.v.shape[-1] == 0:
            m = torch.zeros(*t.v.shape[:-1], 1, dtype=t.v.dtype, device=t.v.device)
        else:
            m = t.v.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        # e^(t - m): its argument's error and rounding, those of the product
        # with log2(e), of the exponential and of a few factors that rescale
        # the running sum; p does not depend on which m was taken
        x = t.v - m
        x = torch.where(self.alive, x, torch.zeros_like(x))
        ev = torch.where(self.alive, torch.exp(x), torch.zeros_like(x))
        rel = t.e + U * (t.v.abs().masked_fill(~self.alive, 0.0) + 3 * x.abs() + 8)
        e = Bounded(ev, ev * rel)
        s = e.sum(-1, keepdim=True)
        over = torch.where(s.v > 0, 1.0 / s.v, torch.zeros_like(s.v))
        # (rescaling: at most one factor per tile of 16 keys, each with its own error)
        more = U * 4 * (t.v.shape[-1] / 16 + 4)
        self.p = (e * Bounded(over, over * over * s.e)).rounded(more / U)
        self.out_h = (self.p @ self.v).rounded(4)

    def out(self):
        return _back(self.out_h)

    def backward(self, g):
        self.do = _rows(g, 1)
        self.dp = self.do @ self.v.T
        self.delta = (self.do * self.out_h).sum(-1, keepdim=True)
        self.d = self.dp - self.delta
        self.ds = (self.p * self.d).where(self.alive)
        dq = _back((self.ds @ self.k) * self.scale)
        dk = _shared((self.ds.T @ self.q) * self.scale, self.share)
        dv = _shared(self.p.T @ self.do, self.share)
        db = self.ds.sum(2).sum(1)
        return dq, dk, dv, db

    def backward2(self, vq, vk, vv, vb=None):
        a = _rows(vq, 1)
        b, c = (_rows(t.masked_fill(self.dead, 0.0), self.share) for t in (vk, vv))
        G = (a @ self.k.T + self.q @ b.T) * self.scale
        if vb is not None:
            G = G + Bounded(vb.double().masked_fill(~self.alive[:, 0, 0], 0.0)[:, None, None, :])
        G = G.where(self.alive)
        g = (self.p * G).sum(-1, keepdim=True)
        H = (self.p * (G - g)).where(self.alive)
        E = self.do @ c.T
        # (the kernels sum p (G d + E) and take g delta off)
        t = (self.p * (G * self.d + E)).sum(-1, keepdim=True) - g * self.delta
        T = (G * self.d + E) - g * (self.d + self.delta)
        X = (self.p * (T - t)).where(self.alive)
        gdo = _back(H @ self.v + self.p @ c)
        gq = _back((X @ self.k + self.ds @ b) * self.scale)
        gk = _shared((X.T @ self.q + self.ds.T @ a) * self.scale, self.share)
        gv = _shared(H.T @ self.do, self.share)
        gb = X.sum(2).sum(1)
        return gdo, gq, gk, gv, gb


def close(name, got, want):
    """got within 1.01 of want's bound (and of what rounding the result alone takes)."""
    assert got.shape == want.v.shape, f"{name}: shape {tuple(got.shape)}, not {tuple(want.v.shape)}"
    if got.numel() == 0:
        return 0.0
    bound = 1.01 * (want.e + U * want.v.abs()) + 1e-37
    err = (got.detach().double() - want.v).abs()
    assert bool(torch.isfinite(got).all()), f"{name}: {int((~torch.isfinite(got)).sum())} values are not finite"
    worst = float((err / bound).max())
    assert worst <= 1.0, f"{name}: {worst:.3g} times its bound, at most {float(err.max()):.3g} off"
    return worst


# ---- Philox4x32-10, in Python integers ---------------------------------------------

def philox_words(seed, offset, block):
    """The four words of a block, by the published rounds."""
    c = [block & 0xFFFFFFFF, block >> 32 & 0xFFFFFFFF, offset & 0xFFFFFFFF, offset >> 32 & 0xFFFFFFFF]
    k = [seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [b >> 32 ^ c[1] ^ k[0], b & 0xFFFFFFFF, a >> 32 ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [k[0] + 0x9E3779B9 & 0xFFFFFFFF, k[1] + 0xBB67AE85 & 0xFFFFFFFF]
    return c


def kept(seed, offset, elements, p):
    """Whether each of `elements` (numbers) is kept."""
    at = round(p * 2 ** 32)
    return [philox_words(seed, offset, e // 4)[e % 4] >= at for e in elements]
