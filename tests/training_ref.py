"""Plain 64-bit layer norm, dropout and cross entropy with error bounds, for the tests.

As in feed_forward_ref: float64 results from the tensors a kernel read, next to
a bound that counts roundings.  U = 2^-24 is half a step of fp32, HALF[t] half a
step of a tensor's type; a fp32 sum of K terms is off by at most K U times the
sum of their magnitudes, whatever its order.
"""
import numpy as np
import torch

from feed_forward_ref import HALF, U, d


def layer_norm(x, weight, bias, residual, eps, out):
    """dict of (value, bound): y, sum, mean, rstd and, for e4m3, scale (y then in units of the exact scale)."""
    t = x.dtype
    s = d(x) if residual is None else d(x) + d(residual)
    c = s.shape[-1]
    es = 0 if residual is None else U * s.abs()
    mean = s.mean(-1, keepdim=True)
    em = (c + 8) * U * s.abs().mean(-1, keepdim=True)
    apart = s - mean
    ea = em + es + U * apart.abs()                       # of each distance
    var = apart.square().mean(-1, keepdim=True)
    ev = (2 * apart.abs() * ea + ea.square()).mean(-1, keepdim=True) + (c + 16) * U * var
    rstd = 1 / torch.sqrt(var + eps)
    # 1 / sqrt falls ever slower: the lower end of the variance's range is the farther one
    er = 1 / torch.sqrt((var - ev).clamp(min=0) + eps) - rstd + 4 * U * rstd
    w = d(weight)
    b = torch.zeros_like(w) if bias is None else d(bias)
    y = apart * rstd * w + b
    ey = w.abs() * ((rstd + er) * ea + apart.abs() * er + 4 * U * apart.abs() * rstd) + U * y.abs()
    got = {"sum": (s, es + HALF[t] * s.abs() + 1e-38), "mean": (mean[:, 0], em[:, 0] + 1e-38),
           "rstd": (rstd[:, 0], er[:, 0])}
    if out is not torch.float8_e4m3fn:
        got["y"] = (y, ey + HALF[out] * y.abs() + 1e-38)
        return got
    top = y.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    es = ey.amax(-1, keepdim=True) / 448.0 + 2 * U * scale
    got["scale"] = (scale[:, 0], es[:, 0])
    v = y / scale
    ev = ey / scale + v.abs() * (es / scale) + 4 * U * v.abs()
    got["y"] = (v, ev + HALF[out] * v.abs() + 2.0 ** -10)          # normal numbers' half step, or the subnormals'
    return got


def layer_norm_backward(dy, s, weight, mean, rstd, dsum):
    """((dx, bound), (dweight, bound), (dbias, bound))"""
    t = dy.dtype
    dy, s, w = d(dy), d(s), d(weight)
    mean, r = d(mean).reshape(-1, 1), d(rstd).reshape(-1, 1)
    m, c = s.shape
    u = (s - mean) * r
    g = dy * w
    level, along = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
    dx = r * (g - level - u * along)
    e = r * ((c + 16) * U * (g.abs().mean(1, keepdim=True) + u.abs() * (g * u).abs().mean(1, keepdim=True))
             + 8 * U * (g.abs() + level.abs() + (u * along).abs()))
    if dsum is not None:
        dx = dx + d(dsum)
        e = e + U * dx.abs()
    dw, db = (dy * u).sum(0), dy.sum(0)
    edw, edb = (m + 12) * U * (dy * u).abs().sum(0), (m + 8) * U * dy.abs().sum(0)
    return ((dx, e + HALF[t] * dx.abs() + 1e-38), (dw, edw + HALF[t] * dw.abs() + 1e-38),
            (db, edb + HALF[t] * db.abs() + 1e-38))


def lots(count, seed, offset, first=0):
    """The 16-bit numbers of positions first .. first + count (first a multiple of 8): ten rounds of Philox4x32."""
    word, half = np.uint64(0xffffffff), np.uint64(32)
    block = np.arange(first // 8, first // 8 + -(-count // 8), dtype=np.uint64)
    c = [block & word, block >> half, np.full_like(block, offset & 0xffffffff), np.full_like(block, offset >> 32)]
    k = [seed & 0xffffffff, seed >> 32]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xd2511f53), c[2] * np.uint64(0xcd9e8d57)
        c = [(q >> half) ^ c[1] ^ np.uint64(k[0]), q & word, (p >> half) ^ c[3] ^ np.uint64(k[1]), p & word]
        k = [(k[0] + 0x9e3779b9) & 0xffffffff, (k[1] + 0xbb67ae85) & 0xffffffff]
    return np.stack(c, 1).astype("<u4").view("<u2").reshape(-1)[:count].astype(np.int64)


def dropout(x, p, seed, offset, residual):
    """((y, bound), kept)"""
    least = int(np.rint(p * 65536))
    kept = torch.from_numpy(lots(x.numel(), seed, offset) >= least).reshape(x.shape)
    scale = 65536.0 / (65536 - least) if least < 65536 else 0.0
    y = torch.where(kept, d(x) * scale, torch.zeros((), dtype=torch.float64))
    e = 2 * U * y.abs()
    if residual is not None:
        y = y + d(residual)
        e = e + U * y.abs()
    return (y, e + HALF[x.dtype] * y.abs()), kept


# ---------------------------------------------------------------- cross entropy
#
# On the device of the tensors.  The exponential is within 2^-21 (1 + its
# argument's size) of itself (bf16: the argument's rounding), the sums of a row
# are joined in trees: a lane's terms, lanes, 32 lanes of runs, at most DEPTH +
# classes / 1000 additions one after the other.

DEPTH = 96
EXP = 2.0 ** -21


def logits(x, w, bias):
    """(z, bound)"""
    x, w = x.double(), w.double()
    z = x @ w.t()
    e = (x.shape[1] + 8) * U * (x.abs() @ w.abs().t())
    if bias is not None:
        z = z + bias.double()
        e = e + U * torch.where(z.isfinite(), z.abs() + bias.double().abs(), torch.zeros_like(z))
    return z, e


def cross_entropy(x, w, bias, target, reduction, ignore=-100, a=0.0):
    """dict of (value, bound): loss, lse"""
    z, ez = logits(x, w, bias)
    n = z.shape[1]
    top = z.amax(1, keepdim=True)
    p = torch.softmax(z, 1)
    lse = torch.logsumexp(z, 1)
    below = torch.where(p > 0, top - z, torch.zeros_like(z))
    e_log = (p * ez).sum(1) + (DEPTH + n / 1000) * U + EXP * (1 + (p * below).sum(1))
    e_lse = e_log + 4 * U * (lse.abs() + top[:, 0].abs())
    counts = target != ignore
    at = torch.where(counts, target, torch.zeros_like(target))[:, None]
    zt, et = z.gather(1, at)[:, 0], ez.gather(1, at)[:, 0]
    each = lse - (1 - a) * zt
    e = e_log + et + 4 * U * ((lse - top[:, 0]).abs() + (top[:, 0] - zt).abs())
    if a:
        each = each - a * z.mean(1)
        e = e + a * (ez.mean(1) + (DEPTH + n / 1000) * U * z.abs().mean(1)) + 4 * U * (top[:, 0].abs() + z.abs().mean(1))
    each, e = torch.where(counts, each, torch.zeros_like(each)), torch.where(counts, e, torch.zeros_like(e))
    e = e + U * each.abs() + 1e-38
    if reduction != "none":
        m = each.numel()
        total, e_total = each.sum(), e.sum() + (m / 1024 + 32) * U * each.abs().sum()
        many = float(counts.sum()) if reduction == "mean" else 1.0
        each, e = total / many, e_total / many + 2 * U * total.abs() / many
    return {"loss": (each, e), "lse": (lse, e_lse + 1e-38)}


def cross_entropy_backward(dloss, x, w, bias, target, lse, count, ignore=-100, a=0.0):
    """((dx, bound), (dw, bound), (dbias, bound))"""
    t = x.dtype
    z, ez = logits(x, w, bias)
    n = z.shape[1]
    counts = target != ignore
    g = torch.where(counts, dloss.double().reshape(-1), torch.zeros((), dtype=torch.float64, device=z.device))[:, None]
    if count is not None:
        g = g / count.double()
    away = z - lse.double()[:, None]
    p = away.exp()
    goal = torch.full_like(z, a / n)
    goal.scatter_add_(1, torch.where(counts, target, torch.zeros_like(target))[:, None], torch.full_like(z[:, :1], 1 - a))
    far = torch.where(p > 0, away.abs(), torch.zeros_like(away))
    dz = (p - goal) * g
    edz = g.abs() * (p * (ez * 1.01 + U * far + EXP * (1 + far)) + 4 * U * (p + goal)) + 3 * U * dz.abs()
    # an exponential below fp32's least normal number, 2^-126 = 1.18e-38, is 0, and so is a product with one: e^z of -88
    # to -103 would still be a subnormal, so that dz may miss up to 2^-126 (|g| + 1), whatever its own size
    edz = edz + HALF[t] * (dz.abs() + edz) + 2.0 ** -126 * (g.abs() + 1)

    def product(a, ea, b):
        y = a @ b
        return y, (a.shape[1] + 8) * U * ((a.abs() + ea) @ b.abs()) + ea @ b.abs() + HALF[t] * y.abs() + 1e-38

    db = dz.sum(0)
    edb = (dz.shape[0] + 8) * U * dz.abs().sum(0) + edz.sum(0) + HALF[t] * db.abs() + 1e-38
    return product(dz, edz, w.double()), product(dz.t(), edz.t(), x.double()), (db, edb)


def check(got, want, what=""):
    value, bound = want
    got = got.double().reshape(value.shape)
    assert torch.isfinite(got).all(), "%s: not finite" % what
    over = (got - value).abs() - bound
    if over.numel():
        i = int(over.argmax())
        assert float(over.max()) <= 0, "%s: %.9g, expected %.9g +- %.3g (element %d of %s)" % (
            what, float(got.reshape(-1)[i]), float(value.reshape(-1)[i]), float(bound.reshape(-1)[i]), i, tuple(value.shape))
