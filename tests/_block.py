"""64-bit references of the block operators and the error bounds of their
arithmetic (torch, any device).

Every bound is first order and elementwise.  With u = eps / 2 of the 16-bit
type (half a step: bf16 2^-8, f16 2^-11) and G(K) = (K + 8) 2^-23 for an fp32
sum of K products whose additions may truncate (one step each):
  a rounding to 16 bits moves v by at most u |v| (plus the type's smallest step),
  a product of K terms by at most G(K) sum |x| |w|,
  an activation, whose exp2 argument is rounded once, by (|z| + 4)^2 2^-21."""
from __future__ import annotations

import math

import torch

FNS = ("none", "relu", "sqrelu", "sigmoid", "silu", "gelu", "gelu_tanh")
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38, torch.float32: 1e-38}


def f(fn, z):
    if fn == "none":
        return z.clone()
    if fn == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if fn == "sqrelu":
        return torch.where(z < 0, torch.zeros_like(z), z * z)
    if fn == "sigmoid":
        return torch.sigmoid(z)
    if fn == "silu":
        return z * torch.sigmoid(z)
    if fn == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def df(fn, z):
    if fn == "none":
        return torch.ones_like(z)
    if fn == "relu":
        return (z > 0).to(z.dtype)
    if fn == "sqrelu":
        return torch.where(z < 0, torch.zeros_like(z), 2 * z)
    p = torch.sigmoid(z)
    if fn == "sigmoid":
        return p * (1 - p)
    if fn == "silu":
        return p * (1 + z * (1 - p))
    if fn == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def lip(fn, z, e):
    """|f'| near z (within e)."""
    if fn == "sqrelu":
        return 2 * (torch.clamp(z, min=0) + e)
    return torch.full_like(z, 1.2)


def act_err(fn, z):
    """Error of the evaluated activation or its derivative, beside its argument's."""
    if fn in ("none", "relu"):
        return torch.zeros_like(z)
    return (z.abs().clamp(max=100) + 4) ** 2 * 2.0 ** -21


def G(K):
    return (K + 8) * 2.0 ** -23


def rnd(v, dt):
    return U[dt] * v.abs() + TINY[dt]


def D(t):
    return None if t is None else t.double()


def proj(x, w, b):
    """(x w^T + b, its error bound)"""
    x, w = x.double(), w.double()
    z, m = x @ w.T, x.abs() @ w.abs().T
    if b is not None:
        z, m = z + b.double(), m + b.double().abs()
    return z, G(x.shape[1]) * m


def linear(x, w, b, fn, scale, r, out_dt):
    """{name: (value, bound)} of z and y."""
    z, ez = proj(x, w, b)
    v = f(fn, z)
    ev = lip(fn, z, ez) * ez + act_err(fn, z)
    y = scale * v + (0 if r is None else r.double())
    e = abs(scale) * ev + 2.0 ** -22 * (abs(scale) * v.abs() + y.abs()) + rnd(y, out_dt)
    return {"z": (z, ez + rnd(z, x.dtype)), "y": (y, e)}


def linear_bwd(dy, x, w, z, fn, scale, grad_dt):
    dt = x.dtype
    dy, x, w = dy.double(), x.double(), w.double()
    zz = dy if z is None else z.double()
    dz = scale * dy * df(fn, zz)
    # dz is rounded to 16 bits before the products; its sums are not
    e32 = abs(scale) * dy.abs() * act_err(fn, zz) + 2.0 ** -21 * dz.abs()
    e16 = e32 + rnd(dz, dt)
    dx, dw, db = dz @ w, dz.T @ x, dz.sum(0)
    T, N = dz.shape
    return {"dx": (dx, (e16 + G(N) * dz.abs()) @ w.abs() + rnd(dx, dt)),
            "dw": (dw, (e16 + G(T) * dz.abs()).T @ x.abs() + rnd(dw, grad_dt)),
            "db": (db, (e16 + G(T) * dz.abs()).sum(0) + rnd(db, grad_dt))}


def ffn(x, wg, wu, wd, bg, bu, bd, fn):
    dt = x.dtype
    u, eu = proj(x, wu, bu)
    out = {"u": (u, eu + rnd(u, dt))}
    if wg is not None:
        g, eg = proj(x, wg, bg)
        out["g"] = (g, eg + rnd(g, dt))
        fg = f(fn, g)
        ef = lip(fn, g, eg) * eg + act_err(fn, g)
        a, ea = fg * u, ef * u.abs() + fg.abs() * eu + ef * eu
    else:
        a, ea = f(fn, u), lip(fn, u, eu) * eu + act_err(fn, u)
    ea = ea + 2.0 ** -22 * a.abs() + rnd(a, dt)  # a is rounded to 16 bits before its product
    out["a"] = (a, ea)
    wd = wd.double()
    y = a @ wd.T
    m = a.abs() @ wd.abs().T
    if bd is not None:
        y, m = y + bd.double(), m + bd.double().abs()
    out["y"] = (y, ea @ wd.abs().T + G(a.shape[1]) * m + rnd(y, dt))
    return out


def ffn_bwd(dy, x, wg, wu, wd, g, u, a, fn, grad_dt):
    dt = x.dtype
    dy, x, wu, wd, u = map(D, (dy, x, wu, wd, u))
    da = dy @ wd
    eda = G(wd.shape[0]) * (dy.abs() @ wd.abs())
    gr = {}
    if wg is not None:
        wg, g = wg.double(), g.double()
        parts = [("gate", da * u * df(fn, g), u.abs() * (eda * df(fn, g).abs() + da.abs() * act_err(fn, g)), wg),
                 ("up", da * f(fn, g), eda * f(fn, g).abs() + da.abs() * act_err(fn, g), wu)]
    else:
        parts = [("up", da * df(fn, u), eda * df(fn, u).abs() + da.abs() * act_err(fn, u), wu)]
    T, n = u.shape
    dx, edx = 0, 0
    for name, v, e, w in parts:
        e = e + 2.0 ** -21 * v.abs() + rnd(v, dt)
        dx, edx = dx + v @ w, edx + (e + G(2 * n) * v.abs()) @ w.abs()
        dw, db = v.T @ x, v.sum(0)
        gr["w_" + name] = (dw, (e + G(T) * v.abs()).T @ x.abs() + rnd(dw, grad_dt))
        gr["b_" + name] = (db, (e + G(T) * v.abs()).sum(0) + rnd(db, grad_dt))
    gr["dx"] = (dx, edx + rnd(dx, dt))
    if a is not None:
        dwd = dy.T @ a.double()
        gr["w_down"] = (dwd, G(T) * (dy.abs().T @ a.double().abs()) + rnd(dwd, grad_dt))
    db = dy.sum(0)
    gr["b_down"] = (db, G(T) * dy.abs().sum(0) + rnd(db, grad_dt))
    return gr


# ------------------------------------------------------------------ norms
# A row's sums add at most 32 values per thread and then a tree of 10 levels:
# under 64 roundings, each 2^-24, so statistics are within 2^-18 relative;
# C covers that and the few roundings per element.
C = 2.0 ** -17


def hat(kind, v, eps):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    return v * r, r


def gate_rows(gate, T, rows):
    g = gate.double()
    return g if rows == 0 else g[torch.arange(T, device=g.device) // rows]


def _norm(kind, v, ev, w, b, eps):
    """(norm, bound) of rows v known to within ev"""
    h, r = hat(kind, v, eps)
    spread = v.abs() + (v.abs().mean(1, keepdim=True) if kind == "layer" else 0)
    e = r * (C * spread + ev + ev.mean(1, keepdim=True)) + h.abs() * r * (ev * h.abs()).mean(1, keepdim=True)
    w = 1 if w is None else w.double()
    out = h * w
    e = e * (w.abs() if torch.is_tensor(w) else 1) + C * out.abs()
    if b is not None:
        out, e = out + b.double(), e + C * b.double().abs()
    return out, e


def norm_fwd(x, y, gate, rows, pre, post, wp, bp, wq, bq, rs, bs, eps, dt):
    T = x.shape[0]
    xo = rs * x.double()
    e = 2.0 ** -22 * xo.abs()
    if y is not None:
        v, ev = y.double(), torch.zeros_like(y, dtype=torch.float64)
        if post != "none":
            v, ev = _norm(post, v, ev, wq, bq, eps)
        g = bs * (gate_rows(gate, T, rows) if gate is not None else torch.ones_like(v))
        xo = xo + g * v
        e = e + g.abs() * ev + 2.0 ** -22 * ((g * v).abs() + xo.abs())
    out = {"x": (xo, e + rnd(xo, x.dtype))}
    if pre != "none":
        h, eh = _norm(pre, xo, e, wp, bp, eps)
        out["h"] = (h, eh + rnd(h, dt))
    return out


def norm_bwd(dxo, dh, xo, y, gate, rows, pre, post, wp, wq, bq, rs, bs, eps, dt, grad_dt):
    """{name: (value, bound)}; a bound of the statistics' kind scales every
    term of a formula by C."""
    T = xo.shape[0]
    mean = lambda v: v.mean(1, keepdim=True)
    out = {}
    Dv = torch.zeros_like(xo, dtype=torch.float64) if dxo is None else dxo.double()
    E = 2.0 ** -22 * Dv.abs()
    if pre != "none":
        xh, r = hat(pre, xo.double(), eps)
        ex = C * (xh.abs() + r * mean(xo.double().abs()))
        w = torch.ones_like(xh[0]) if wp is None else wp.double()
        q = dh.double() * w
        c1, c2 = (mean(q) if pre == "layer" else 0 * mean(q)), mean(q * xh)
        m1, m2 = mean(q.abs()), mean((q * xh).abs())
        Dv = Dv + r * (q - c1 - xh * c2)
        E = E + C * r * (q.abs() + m1 + xh.abs() * m2) * 2 + r * (ex * m2 + xh.abs() * mean(q.abs() * ex))
        dh_ = dh.double()
        v = (dh_ * xh).sum(0)
        out["w_pre"] = (v, (dh_.abs() * (ex + G(T) * xh.abs())).sum(0) + rnd(v, grad_dt))
        v = dh_.sum(0)
        out["b_pre"] = (v, G(T) * dh_.abs().sum(0) + rnd(v, grad_dt))
    E = E + 2.0 ** -22 * Dv.abs()
    out["dx"] = (rs * Dv, abs(rs) * E + 2.0 ** -23 * abs(rs) * Dv.abs() + rnd(rs * Dv, xo.dtype))
    if y is None:
        return out
    y = y.double()
    g = bs * (gate_rows(gate, T, rows) if gate is not None else torch.ones_like(y))
    w = torch.ones_like(y[0]) if wq is None or post == "none" else wq.double()
    b = torch.zeros_like(y[0]) if bq is None or post == "none" else bq.double()
    if post == "none":
        yh, r, ey = y, 1.0, torch.zeros_like(y)
        dy, edy = g * Dv, g.abs() * E
    else:
        yh, r = hat(post, y, eps)
        ey = C * (yh.abs() + r * mean(y.abs()))
        q, eq = g * Dv * w, (g * w).abs() * (E + C * Dv.abs())
        c1, c2 = (mean(q) if post == "layer" else 0 * mean(q)), mean(q * yh)
        m1, m2 = mean(q.abs()), mean((q * yh).abs())
        dy = r * (q - c1 - yh * c2)
        edy = r * (eq + mean(eq) + yh.abs() * mean(eq * yh.abs()) + 2 * C * (q.abs() + m1 + yh.abs() * m2) + ey * m2 +
                   yh.abs() * mean(q.abs() * ey))
    out["dy"] = (dy, edy + 2.0 ** -22 * dy.abs() + rnd(dy, dt))
    v, ev = yh * w + b, ey * w.abs() + 2.0 ** -22 * ((yh * w).abs() + b.abs())
    if gate is not None:
        n = gate.shape[0]
        at = torch.zeros(T, dtype=torch.long, device=y.device) if rows == 0 else torch.arange(T, device=y.device) // rows
        add = lambda t: torch.zeros(n, y.shape[1], dtype=torch.float64, device=y.device).index_add_(0, at, t)
        val = bs * add(Dv * v)
        mag = (Dv * yh * w).abs() + (Dv * b).abs()  # w S1 and b S0 are summed apart
        out["gate"] = (val, abs(bs) * add(E * (v.abs() + (yh * w).abs() + b.abs()) + Dv.abs() * ev + G(T) * mag) +
                       rnd(val, grad_dt))
    if post != "none":
        s = (g * Dv * yh).sum(0)
        out["w_post"] = (s, (g.abs() * (E * yh.abs() + Dv.abs() * ey + G(T) * (Dv * yh).abs())).sum(0) + rnd(s, grad_dt))
        s = (g * Dv).sum(0)
        out["b_post"] = (s, (g.abs() * (E + G(T) * Dv.abs())).sum(0) + rnd(s, grad_dt))
    return out


def check(got, want, what=""):
    """got within its bound of want = (value, bound)"""
    value, bound = want
    assert got.shape == value.shape, f"{what}: {tuple(got.shape)} vs {tuple(value.shape)}"
    err = (got.double() - value).abs()
    worst = (err - bound).max().item() if err.numel() else -1.0
    if not worst <= 0.0:  # (a NaN fails)
        i = int((err - bound).nan_to_num(nan=math.inf).argmax())
        raise AssertionError(f"{what}: off by {err.flatten()[i]:.3g}, bound {bound.flatten()[i]:.3g}, value "
                             f"{value.flatten()[i]:.6g} at {i} of {tuple(value.shape)}")
