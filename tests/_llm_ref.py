"""Plain 64-bit forms of the 4-bit and gated feed-forward operators, and what their kernels' arithmetic
may lose, for the tests.

Roundings: a value rounded to a type is off by at most half a step, ``finfo.eps / 2`` relative (and half the
smallest subnormal near zero).  A sum of L terms held in fp32, added in any order with additions that lose at
most 2^-23 of their result (the tensor cores may truncate), is off by at most L 2^-23 of the sum of the terms'
magnitudes.
"""
import math

import torch

ACTS = ("silu", "gelu", "gelu_tanh", "relu2")
U = 2.0 ** -23


def act64(name, g):
    """Activation and derivative in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    r = g.clamp(min=0)
    return r * r, 2 * r


def act_slope(name, g):
    """A bound on |act'| near g (the derivatives of the first three stay below 1.13)."""
    return 2 * g.abs() if name == "relu2" else torch.full_like(g, 1.13)


def act_slope2(name, g):
    """A bound on |act''| (1/2, 2 / sqrt(2 pi), its tanh form, 2)."""
    return {"silu": 0.5, "gelu": 0.8, "gelu_tanh": 0.85, "relu2": 2.0}[name]


def act_eps(g):
    """Relative error of the kernels' activation in fp32 arithmetic: the argument of the exponential or of
    erfc, up to 1.6 |g| + 0.08 |g|^3 or g^2 / 2, carries a few 2^-24 of itself into the exponent, the
    functions and the products a few ulp more."""
    a = g.abs()
    return (8 + 2 * a + 2 * a * a + a ** 3) * 2.0 ** -22


def half_step(dtype, v):
    """What one rounding of v to dtype may lose."""
    f = torch.finfo(dtype)
    return v.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def gated_bound(act, g, u, dg, du):
    """Error of act(g) u in fp32 when g and u are off by dg and du."""
    a = act64(act, g)[0]
    da = (act_slope(act, g) + act_slope2(act, g) * dg) * dg + act_eps(g) * a.abs()
    return da * (u.abs() + du) + a.abs() * du + U * (a * u).abs()


def quantize64(a, group, affine):
    """(codes 0..15, scales, offsets or None, values) of the 4-bit format, group by group, in 64 bits."""
    a = a.double()
    m, n = a.shape
    codes, scales, offs, vals = [], [], [], []
    for k in range(0, n, group):
        x = a[:, k:k + group]
        if affine:
            mn, mx = x.amin(1), x.amax(1)
            s = ((mx - mn) / 15).float().half()
            b = (mn + 8 * s.double()).float().half()
        else:
            s = (x.abs().amax(1) / 7).float().half()
            b = torch.zeros_like(s)
        sd, bd = s.double()[:, None], b.double()[:, None]
        q = torch.where(sd > 0, torch.round((x - bd) / torch.where(sd > 0, sd, 1.0)), 0.0).clamp(-8, 7)
        codes.append(q + 8)
        scales.append(s)
        offs.append(b)
        vals.append(sd * q + bd)
    return (torch.cat(codes, 1).to(torch.uint8), torch.stack(scales), torch.stack(offs) if affine else None,
            torch.cat(vals, 1))
