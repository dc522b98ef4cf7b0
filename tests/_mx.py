"""64-bit references of the microscaled operators and the error bounds of
their arithmetic (torch, any device); see tests/_block.py for the bounds of
sums, activations and roundings.

Quantisation of given values is exact arithmetic, so those results are compared
for equality.  Where a kernel quantises what it has computed, known to within e,
its result lies between the quantised ends of [v - e, v + e] under each scale
that an amax within that reach can give (rounding is monotone): the bound."""
from __future__ import annotations

import torch

from tests import _block as R

MX8, MX4 = 4, 5


def pow2(e):
    """2^e in 64 bits, exactly, for -1022 <= e <= 1023 (a library's power may be off by a step)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def table(kind):
    """The type's values from 0 up, by their codes."""
    if kind == MX4:
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    c = torch.arange(127)  # (0x7f is NaN)
    e, m = (c >> 3).double(), (c & 7).double()
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7))


def nearest(kind, a):
    """Codes of the values nearest to a >= 0, of two as near the even code."""
    t = table(kind).to(a.device)
    mid = (t[1:] + t[:-1]) / 2
    lo = torch.bucketize(a, mid)            # values of mid below a
    tie = (lo < mid.numel()) & (mid[lo.clamp(max=mid.numel() - 1)] == a) & (lo % 2 == 1)
    return lo + tie


def scale_exp(kind, amax):
    """The exponent of a block's scale: the least at which amax / 2^e fits."""
    most = table(kind)[-1].item()
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -200) / most))
    e = torch.where(most * pow2(e) < amax, e + 1, e)     # (the logarithm's rounding)
    e = torch.where(most * pow2(e - 1) >= amax, e - 1, e)
    return e.clamp(min=-127)


def blocks(v):
    """[T][K] -> [T][blocks][32], zeros past the row, up to 128 columns"""
    T, K = v.shape
    return torch.nn.functional.pad(v, (0, -K % 128)).reshape(T, -1, 32)


def quantize(kind, v):
    """(codes per column [T][Kp], scale codes [T][blocks], values [T][K]) of 64-bit v; NaN blocks as the library writes them"""
    b = blocks(v)
    amax = b.abs().amax(2)
    bad = ~torch.isfinite(amax)
    e = scale_exp(kind, torch.where(bad, 1.0, amax))
    s = pow2(e)
    q = nearest(kind, torch.where(bad[..., None], 0.0, b).abs() / s[..., None])
    val = table(kind).to(v.device)[q] * s[..., None] * torch.where(torch.signbit(b), -1.0, 1.0)
    sign = torch.signbit(b).long() << (7 if kind == MX8 else 3)
    codes = torch.where(bad[..., None], 0x7f if kind == MX8 else 0, q + sign)
    val = torch.where(bad[..., None], torch.nan, val)
    sc = torch.where(bad, 255, e.long() + 127)
    T, K = v.shape
    return codes.reshape(T, -1), sc, val.reshape(T, -1)[:, :K]


def unpack(q):
    """(codes per column [T][Kp], scale codes [T][blocks]) that an MxMatrix holds, and whether what pads the rows is 0"""
    c = q.codes.long()
    if q.kind == MX4:
        c = torch.stack((c & 15, c >> 4), 2).reshape(c.shape[0], -1)
    Rt, B = q.scales.shape[:2]
    s = q.scales.permute(0, 3, 2, 1, 4).reshape(Rt * 128, B * 4).long()
    T = c.shape[0]
    return c, s[:T], bool((s[T:] == 0).all())


def values(q):
    """What an MxMatrix stands for, 64-bit."""
    c, s, _ = unpack(q)
    top = 128 if q.kind == MX8 else 8
    t = torch.cat((table(q.kind), torch.tensor([torch.nan], dtype=torch.float64))) if q.kind == MX8 else table(q.kind)
    v = t.to(c.device)[c % top] * torch.where(c >= top, -1.0, 1.0)
    sc = torch.where(s == 255, torch.nan, pow2(s - 127))
    return (v.reshape(c.shape[0], -1, 32) * sc[..., None]).reshape(c.shape[0], -1)[:, : q.cols]


def requantized(kind, v, e):
    """(value, bound) of the quantised v that is known to within e."""
    T, K = v.shape
    b, eb = blocks(v), blocks(e)
    amax, reach = b.abs().amax(2), eb.amax(2)
    val = quantize(kind, v)[2]
    full = blocks(val)
    bound = torch.zeros_like(b)
    for am in ((amax - reach).clamp(min=0), amax + reach):
        s = pow2(scale_exp(kind, am))[..., None]
        most = table(kind)[-1].item()
        for end in (b - eb, b + eb):
            x = end / s
            q = table(kind).to(v.device)[nearest(kind, x.abs().clamp(max=most))] * torch.sign(x) * s
            bound = torch.maximum(bound, (q - full).abs())
    return val, bound.reshape(T, -1)[:, :K]


def proj(x, w, b):
    z, m = x @ w.T, x.abs() @ w.abs().T
    if b is not None:
        z, m = z + b.double(), m + b.double().abs()
    return z, R.G(x.shape[1]) * m


def linear(x, w, b, fn, scale, r, out_dt):
    z, ez = proj(values(x), values(w), b)
    v = R.f(fn, z)
    ev = R.lip(fn, z, ez) * ez + R.act_err(fn, z)
    y = scale * v + (0 if r is None else r.double())
    return y, abs(scale) * ev + 2.0 ** -22 * (abs(scale) * v.abs() + y.abs()) + R.rnd(y, out_dt)


def ffn(x, wg, wu, wd, bg, bu, bd, fn, dt):
    xv = values(x)
    u, eu = proj(xv, values(wu), bu)
    if wg is not None:
        g, eg = proj(xv, values(wg), bg)
        fg = R.f(fn, g)
        ef = R.lip(fn, g, eg) * eg + R.act_err(fn, g)
        a, ea = fg * u, ef * u.abs() + fg.abs() * eu + ef * eu
    else:
        a, ea = R.f(fn, u), R.lip(fn, u, eu) * eu + R.act_err(fn, u)
    a, ea = requantized(x.kind, a, ea + 2.0 ** -22 * a.abs())
    wdv = values(wd)
    y, m = a @ wdv.T, a.abs() @ wdv.abs().T
    if bd is not None:
        y, m = y + bd.double(), m + bd.double().abs()
    return y, ea @ wdv.abs().T + R.G(a.shape[1]) * m + R.rnd(y, dt)
