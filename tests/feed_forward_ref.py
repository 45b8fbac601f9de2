"""Plain 64-bit feed-forward operators with error bounds, for the tests.

Every function takes the tensors a kernel read (any type) and returns float64
results next to a bound on how far a kernel's outputs may be from them.  The
bounds count roundings:

  u = 2^-24 is half a step of fp32, HALF[t] half a step of the output type.
  A sum of K products in fp32, in any order, is off by at most K u times the
  sum of the products' magnitudes (here (K + 8) u: a few more for scales and
  bias).
  Activations and their slopes: |act'| <= 1.13 carries an error of z over; the
  exponential, its argument's rounding and the reciprocal are within 2^-20
  (1 + |z|) relative to |z| + |value|; the e4m3 and bf16 GELU's distribution
  function is within 1.5e-7 < 2^-22, covered by the same term.
  dz enters a product rounded to the tensors' type: HALF[t] |dz|.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
ACT_ERR = 2.0 ** -20
LIP = 1.13


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def slope(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def d(t):
    return None if t is None else t.detach().cpu().double()


def _act_error(z, ez, name):
    if name == "none":
        return ez
    if name == "relu":
        return ez
    return LIP * ez + ACT_ERR * (z.abs() + act(z, name).abs()) * (1 + z.abs())


def product(x, w, xs=None, ws=None):
    """(x w^T, bound) for a fp32 sum."""
    x, w = d(x), d(w)
    if xs is not None:
        x, w = x * d(xs).reshape(-1, 1), w * d(ws).reshape(-1, 1)
    return x @ w.t(), (x.shape[1] + 8) * U * (x.abs() @ w.abs().t())


def linear(x, w, bias, residual, name, out, xs=None, ws=None):
    """((y, bound), (z, bound))"""
    z, ez = product(x, w, xs, ws)
    if bias is not None:
        z = z + d(bias)
        ez = ez + U * (z.abs() + d(bias).abs())
    y, ey = act(z, name), _act_error(z, ez, name)
    if residual is not None:
        y = y + d(residual)
        ey = ey + U * y.abs()
    return (y, ey + HALF[out] * y.abs() + 1e-38), (z, ez + HALF[out] * z.abs() + 1e-38)


def gated(x, wg, wu, name, out, xs=None, gs=None, us=None):
    """((y, bound), (gate, bound), (up, bound))"""
    g, eg = product(x, wg, xs, gs)
    u, eu = product(x, wu, xs, us)
    a, ea = act(g, name), _act_error(g, eg, name)
    y = a * u
    ey = ea * u.abs() + a.abs() * eu + ea * eu + U * y.abs() + HALF[out] * y.abs() + 1e-38
    return (y, ey), (g, eg + HALF[out] * g.abs() + 1e-38), (u, eu + HALF[out] * u.abs() + 1e-38)


def _sum(a, ea, b, out):
    """a b with a off by ea: (value, bound)."""
    y = a @ b
    return y, (a.shape[1] + 8) * U * ((a.abs() + ea) @ b.abs()) + ea @ b.abs() + HALF[out] * y.abs() + 1e-38


def linear_backward(dy, x, w, z, name):
    """((dx, bound), (dw, bound), (dbias, bound))"""
    t = dy.dtype
    dy, x, w = d(dy), d(x), d(w)
    dz, soft = dy, torch.zeros_like(dy)
    if name != "none":
        z = d(z)
        dz = dy * slope(z, name)
        if name != "relu":
            soft = ACT_ERR * dy.abs() * (1 + z.abs())
    edz = soft + (HALF[t] * (dz.abs() + soft) if name != "none" else 0)
    dx = _sum(dz, edz, w, t)
    dw = _sum(dz.t(), edz.t(), x, t)
    db = dz.sum(0)
    edb = (dz.shape[0] + 8) * U * dz.abs().sum(0) + soft.sum(0) + HALF[t] * db.abs() + 1e-38
    return dx, dw, (db, edb)


def gated_backward(dy, x, wg, wu, gate, up, name):
    """((dx, bound), (dw_gate, bound), (dw_up, bound))"""
    t = dy.dtype
    dy, x, wg, wu, g, u = d(dy), d(x), d(wg), d(wu), d(gate), d(up)
    dg = dy * u * slope(g, name)
    du = dy * act(g, name)
    hard = name in ("none", "relu")
    sg = (0 if hard else ACT_ERR) * (dy * u).abs() * (1 + g.abs()) + 2 * U * dg.abs()
    su = (0 if hard else ACT_ERR) * dy.abs() * (g.abs() + act(g, name).abs()) * (1 + g.abs()) + 2 * U * du.abs()
    eg, eu = sg + HALF[t] * (dg.abs() + sg), su + HALF[t] * (du.abs() + su)
    both, eboth = torch.cat([dg, du], 1), torch.cat([eg, eu], 1)
    dx = _sum(both, eboth, torch.cat([wg, wu], 0), t)
    return dx, _sum(dg.t(), eg.t(), x, t), _sum(du.t(), eu.t(), x, t)


def rms_norm(x, weight, residual, eps, out):
    """dict of (value, bound): y, sum, rstd and, for e4m3, scale (y then in units of the exact scale)."""
    t = x.dtype
    s = d(x) if residual is None else d(x) + d(residual)
    c = s.shape[-1]
    rstd = 1 / torch.sqrt((s * s).mean(-1) + eps)
    y = s * rstd[:, None] * d(weight)
    er = (c + 16) * U                                    # relative, of rstd and of what follows it
    got = {"sum": (s, (U + HALF[t]) * s.abs() + 1e-38), "rstd": (rstd, er * rstd)}
    if out is not torch.float8_e4m3fn:
        got["y"] = (y, (er + HALF[out]) * y.abs() + 1e-38)
        return got
    top = y.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    got["scale"] = (scale, 2 * er * scale)
    v = y / scale[:, None]
    got["y"] = (v, (4 * er + HALF[out]) * v.abs() + 2.0 ** -10)   # normal numbers' half step, or the subnormals'
    return got


def rms_norm_backward(dy, s, weight, rstd, dsum):
    """((dx, bound), (dweight, bound))"""
    t = dy.dtype
    dy, s, w, r = d(dy), d(s), d(weight), d(rstd).reshape(-1, 1)
    c, m = s.shape[1], s.shape[0]
    g = dy * w
    mean = (g * s).mean(1, keepdim=True)
    dx = r * (g - s * r * r * mean)
    e = 16 * U * r * (g.abs() + (s * r * r * mean).abs()) + (c + 16) * U * r * s.abs() * r * r * (g * s).abs().mean(1, keepdim=True)
    if dsum is not None:
        dx = dx + d(dsum)
        e = e + U * dx.abs()
    dw = (dy * s * r).sum(0)
    edw = (m + 8) * U * (dy * s * r).abs().sum(0)
    return (dx, e + HALF[t] * dx.abs() + 1e-38), (dw, edw + HALF[t] * dw.abs() + 1e-38)


def check(got, want, what=""):
    value, bound = want
    got = d(got).reshape(value.shape)
    assert torch.isfinite(got).all(), "%s: not finite" % what
    over = (got - value).abs() - bound
    if over.numel():
        i = int(over.argmax())
        assert float(over.max()) <= 0, "%s: %.9g, expected %.9g +- %.3g (element %d of %s)" % (
            what, float(got.reshape(-1)[i]), float(value.reshape(-1)[i]), float(bound.reshape(-1)[i]), i,
            tuple(value.shape))
