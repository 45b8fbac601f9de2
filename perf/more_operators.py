"""The operators around a trained feed-forward network: cases, inputs, plain forms and 64-bit results.

  norm     s = x + residual, y = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias, y in x's type or in e4m3 with a
           scale per row
  dropout  y = x / (1 - p) where a random number of the element's position says so, else 0, + residual
  loss     the cross entropy of softmax(x W^T + bias) against one class per row

``run`` computes a case either with the library's entry points (``own``) or in plain torch, in 32 bits.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": F8}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1}
IGNORE = -100
WORD = 0xffffffff

# The widths are the library's own fully-connected ones: 4096 features, 9216 = 256 x 6 x 6 in the wide layer, 1000
# classes; larger numbers of classes are a language's vocabulary.


def listed():
    return [
        # one token's norm between two layers while serving: launch latency
        norm("norm_token", 1, 4096, "bf16", "bf16", True),
        # a long prompt's norm, quantised by rows for an 8-bit product
        norm("norm_prompt_e4m3", 4095, 4096, "bf16", "e4m3", True),
        # rows of an odd length in fp32, unaligned: a classifier's 1001 outputs normalised
        norm("norm_odd_f32", 1023, 1001, "f32", "f32", False),
        # a training step's norm gradient, the weight's and the bias's with it
        norm("norm_train_backward", 8192, 4096, "bf16", "bf16", True, backward=True),
        # AlexNet's dropout behind fc6: half of 128 images' 4096 features, a small call
        dropout("dropout_fc6", 128, 4096, "f32", 0.5, False),
        # a sublayer's output on its way into the residual stream
        dropout("dropout_rows", 8192, 4096, "bf16", 0.1, True),
        # the gradient in the wide layer, odd row count
        dropout("dropout_wide_backward", 4095, 9216, "bf16", 0.1, False, backward=True),
        # one token scored against a vocabulary: the weights stream once from memory
        loss("loss_token", 1, 65536, 4096, "bf16", False, "none", 0.0, False),
        # the loss of AlexNet's fc8 in its own type
        loss("loss_fc8_f32", 128, 1000, 4096, "f32", True, "mean", 0.0, False),
        # a classifier's training step with smoothed labels
        loss("loss_fc8_backward", 256, 1000, 4096, "bf16", True, "mean", 0.1, False, backward=True),
        # a packed batch's loss over a vocabulary of odd size, padding ignored
        loss("loss_rows", 4096, 50021, 4096, "bf16", False, "mean", 0.0, True),
        # its gradients
        loss("loss_train_backward", 4096, 50021, 4096, "bf16", False, "mean", 0.0, True, backward=True),
    ]


def norm(name, m, c, dtype, out, residual, backward=False):
    return {"name": name, "op": "norm", "m": m, "c": c, "dtype": dtype, "out": out, "residual": residual,
            "backward": backward}


def dropout(name, m, c, dtype, p, residual, backward=False):
    return {"name": name, "op": "dropout", "m": m, "c": c, "dtype": dtype, "p": p, "residual": residual,
            "backward": backward}


def loss(name, m, n, k, dtype, bias, reduction, smoothing, padded, backward=False):
    return {"name": name, "op": "loss", "m": m, "n": n, "k": k, "dtype": dtype, "bias": bias, "reduction": reduction,
            "smoothing": smoothing, "padded": padded, "backward": backward}


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        kind = rng.random()          # mostly whole tiles' multiples, as layers have; odd ones among them
        if kind < 0.4 and v >= 64:
            v -= v % 64
        elif kind < 0.7 and v >= 8:
            v -= v % 8
        return v

    op = rng.choice(["norm", "dropout", "loss", "loss"])
    backward = rng.random() < 0.5
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        out = dtype if backward or rng.random() < 0.6 else "e4m3"
        case = norm("", size(64 if backward else 1, 8192), size(256, 9216), dtype, out, rng.random() < 0.6, backward)
    elif op == "dropout":
        case = dropout("", size(1, 8192), size(256, 9216), rng.choice(["bf16", "bf16", "f32"]),
                       rng.choice([0.1, 0.2, 0.5, round(rng.uniform(0.01, 0.9), 3)]),
                       not backward and rng.random() < 0.6, backward)
    else:
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        n, k = size(1000, 50021), size(256, 4096)
        most = (1 << 39) if dtype == "bf16" else (1 << 36)
        m = max(1, min(size(64 if backward else 1, 4096), most // (n * k)))
        case = loss("", m, n, k, dtype, rng.random() < 0.4, rng.choice(["mean", "mean", "sum", "none"]),
                    rng.choice([0.0, 0.0, 0.1]), m > 16 and rng.random() < 0.5, backward)
    del case["name"]
    return case


def work(case):
    m, e = case["m"], BYTES[case["dtype"]]
    if case["op"] == "norm":
        one = m * case["c"] * e
        if case["backward"]:         # dy, s and the gradient that reaches s directly in, ds out; weight, mean, 1/std in
            return {"bytes": one * (4 if case["residual"] else 3) + 3 * case["c"] * e + 8 * m,
                    "flops": 14.0 * m * case["c"]}
        return {"bytes": one * (3 if case["residual"] else 1) + m * case["c"] * BYTES[case["out"]] + 2 * case["c"] * e
                + (12 if case["out"] == "e4m3" else 8) * m, "flops": 9.0 * m * case["c"]}
    if case["op"] == "dropout":
        return {"bytes": m * case["c"] * e * (3 if case["residual"] else 2), "flops": 2.0 * m * case["c"]}
    n, k = case["n"], case["k"]
    vectors = 12 * m + (n * e if case["bias"] else 0)            # target and a number per row
    if case["backward"]:             # the logits again, then dx and dw
        return {"bytes": 2 * e * (m * k + n * k) + vectors + (n * e if case["bias"] else 0), "flops": 6.0 * m * n * k}
    return {"bytes": e * (m * k + n * k) + vectors, "flops": 2.0 * m * n * k}


# ---------------------------------------------------------------- inputs


def quantise_rows(v):
    """Rows in e4m3 and their scales."""
    scale = v.abs().amax(dim=1) / F8_MAX
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (v / scale[:, None]).clamp(-F8_MAX, F8_MAX).to(F8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=None):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype or dt)

    m = case["m"]
    s = {"case": dict(case)}
    if case["op"] == "norm":
        c = case["c"]
        s["weight"] = normal(c, std=0.1, mean=1.0)
        if case["backward"]:
            s["sum"] = normal(m, c, std=1.5, mean=0.3)
            v = s["sum"].float()
            s["mean"] = v.mean(dim=1)
            s["rstd"] = ((v - s["mean"][:, None]).square().mean(dim=1) + EPS).rsqrt()
            s["dy"] = normal(m, c, std=0.5)
            s["dsum"] = normal(m, c, std=0.5) if case["residual"] else None
        else:
            s["bias"] = normal(c, std=0.1)
            s["x"] = normal(m, c)
            s["residual"] = normal(m, c, std=2.0, mean=0.3) if case["residual"] else None
        return s
    if case["op"] == "dropout":
        s["seed"], s["offset"] = (seed * 0x9e3779b97f4a7c15 + 12345) % (1 << 64), seed % 1000
        s["x"] = normal(m, case["c"])
        s["residual"] = normal(m, case["c"], std=2.0) if case["residual"] else None
        return s
    n, k = case["n"], case["k"]
    s["x"] = normal(m, k)
    s["w"] = normal(n, k, std=2 * k ** -0.5)
    s["bias"] = normal(n, std=0.5) if case["bias"] else None
    # classes as often as words are: a few frequent ones, most hardly ever
    s["target"] = (torch.rand(m, generator=g, device="cuda").pow(3) * n).long().clamp(max=n - 1)
    if case["padded"]:               # the batch's end is padding
        s["target"][m - m // 16:] = IGNORE
    if case["backward"]:
        z = logits_plain(s)
        top = z.amax(dim=1)
        s["lse"] = top + torch.log(torch.exp(z - top[:, None]).sum(dim=1))
        rows = m if case["reduction"] == "none" else 1
        s["dloss"] = torch.rand(rows, generator=g, device="cuda").add_(0.5)
        if rows == 1 and case["reduction"] != "none":
            s["dloss"] = s["dloss"][0]
        s["count"] = (s["target"] != IGNORE).sum().float() if case["reduction"] == "mean" else None
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(s):
    import convolution_forward_conv2d_amd as mic

    case = s["case"]
    if case["op"] == "norm":
        if case["backward"]:
            dx, dweight, dbias = mic.layer_norm_backward(s["dy"], s["sum"], s["weight"], s["mean"], s["rstd"],
                                                         dsum=s["dsum"], bias=True)
            return {"dx": dx, "dweight": dweight, "dbias": dbias}
        r = mic.layer_norm(s["x"], s["weight"], bias=s["bias"], residual=s["residual"], eps=EPS,
                           out_dtype=TYPES[case["out"]])
        out = {"y": r.y, "mean": r.mean, "rstd": r.rstd}
        if case["residual"]:
            out["sum"] = r.sum
        if case["out"] == "e4m3":
            out["scale"] = r.scale
        return out
    if case["op"] == "dropout":
        if case["backward"]:
            return mic.dropout_backward(s["x"], case["p"], s["seed"], offset=s["offset"])
        return mic.dropout(s["x"], case["p"], s["seed"], offset=s["offset"], residual=s["residual"])
    if case["backward"]:
        dx, dw, dbias = mic.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["target"], s["lse"],
                                                          bias=s["bias"], count=s["count"],
                                                          label_smoothing=case["smoothing"])
        return {"dx": dx, "dw": dw, "dbias": dbias} if case["bias"] else {"dx": dx, "dw": dw}
    r = mic.linear_cross_entropy(s["x"], s["w"], s["target"], bias=s["bias"], reduction=case["reduction"],
                                 label_smoothing=case["smoothing"])
    return {"loss": r.loss, "lse": r.lse}


def logits_plain(s):
    z = s["x"].float() @ s["w"].float().t()
    return z if s["bias"] is None else z + s["bias"].float()


def lots_plain(count, seed, offset, device):
    """A 16-bit random number for each of `count` positions: ten rounds of Philox4x32 on the position's eighth."""
    block = torch.arange((count + 7) // 8, device=device)
    c = [block & WORD, block >> 32, torch.full_like(block, offset & WORD), torch.full_like(block, offset >> 32)]
    k0, k1 = seed & WORD, seed >> 32
    for _ in range(10):
        # the product's 64 bits wrap into the sign; both halves come out whole
        p0, p1 = c[0] * 0xd2511f53, c[2] * 0xcd9e8d57
        c = [(p1 >> 32) & WORD ^ c[1] ^ k0, p1 & WORD, (p0 >> 32) & WORD ^ c[3] ^ k1, p0 & WORD]
        k0, k1 = (k0 + 0x9e3779b9) & WORD, (k1 + 0xbb67ae85) & WORD
    return torch.stack([half for word in c for half in (word & 0xffff, word >> 16)], dim=1).reshape(-1)[:count]


def run_plain(s):
    case = s["case"]
    dt = TYPES[case["dtype"]]
    if case["op"] == "norm":
        w = s["weight"].float()
        if case["backward"]:
            dy, rstd = s["dy"].float(), s["rstd"][:, None]
            unit = (s["sum"].float() - s["mean"][:, None]) * rstd
            g = dy * w
            ds = rstd * (g - g.mean(dim=1, keepdim=True) - unit * (g * unit).mean(dim=1, keepdim=True))
            if case["residual"]:
                ds = ds + s["dsum"].float()
            return {"dx": ds.to(dt), "dweight": (dy * unit).sum(dim=0).to(dt), "dbias": dy.sum(dim=0).to(dt)}
        v = s["x"].float()
        if case["residual"]:
            v = v + s["residual"].float()
        mean = v.mean(dim=1)
        apart = v - mean[:, None]
        rstd = 1 / torch.sqrt((apart * apart).mean(dim=1) + EPS)
        y = apart * rstd[:, None] * w + s["bias"].float()
        out = {"mean": mean, "rstd": rstd}
        if case["residual"]:
            out["sum"] = v.to(dt)
        if case["out"] == "e4m3":
            out["y"], out["scale"] = quantise_rows(y)
        else:
            out["y"] = y.to(dt)
        return out
    if case["op"] == "dropout":
        x = s["x"].float()
        least = round(case["p"] * 65536)
        kept = (lots_plain(x.numel(), s["seed"], s["offset"], x.device) >= least).reshape(x.shape)
        y = torch.where(kept, x * (65536 / (65536 - least)), torch.zeros_like(x))
        if case["residual"]:
            y = y + s["residual"].float()
        return y.to(dt)
    n, a = case["n"], case["smoothing"]
    target = s["target"]
    counts = target != IGNORE
    at = torch.where(counts, target, torch.zeros_like(target))
    z = logits_plain(s)
    if case["backward"]:
        g = torch.where(counts, s["dloss"], torch.zeros_like(s["lse"]))
        if case["reduction"] == "mean":
            g = g / s["count"]
        dz = torch.exp(z - s["lse"][:, None])
        if a:
            dz = dz - a / n
        rows = torch.arange(case["m"], device=z.device)
        dz[rows, at] = dz[rows, at] - (1 - a)
        dz = dz * g[:, None]
        out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt)}
        if case["bias"]:
            out["dbias"] = dz.sum(dim=0).to(dt)
        return out
    top = z.amax(dim=1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(dim=1))
    each = lse - (1 - a) * z.gather(1, at[:, None])[:, 0]
    if a:
        each = each - a * z.mean(dim=1)
    each = torch.where(counts, each, torch.zeros_like(each))
    if case["reduction"] == "mean":
        each = each.sum() / counts.sum()
    elif case["reduction"] == "sum":
        each = each.sum()
    return {"loss": each, "lse": lse}


# ---------------------------------------------------------------- the definition in 64 bits


def lots64(count, seed, offset):
    """The same numbers on the host, in unsigned 64-bit integers."""
    word, half = np.uint64(WORD), np.uint64(32)
    block = np.arange(-(-count // 8), dtype=np.uint64)
    a, b = block & word, block >> half
    c, d = np.full_like(block, offset & WORD), np.full_like(block, offset >> 32)
    for i in range(10):
        key0 = np.uint64(((seed & WORD) + i * 0x9e3779b9) & WORD)
        key1 = np.uint64(((seed >> 32) + i * 0xbb67ae85) & WORD)
        first, second = a * np.uint64(0xd2511f53), c * np.uint64(0xcd9e8d57)
        a, b, c, d = (second >> half) ^ b ^ key0, second & word, (first >> half) ^ d ^ key1, first & word
    words = np.stack([a, b, c, d], axis=1).astype("<u4")
    return words.view("<u2").reshape(-1)[:count]


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if case["op"] == "norm":
        w = d["weight"]
        if case["backward"]:
            unit = (d["sum"] - d["mean"].unsqueeze(1)) * d["rstd"].unsqueeze(1)
            # what the norm takes out of a gradient: its parts along the ones and along the row itself
            g = d["dy"] * w
            level = torch.einsum("mc->m", g) / case["c"]
            along = torch.einsum("mc,mc->m", g, unit) / case["c"]
            dx = (g - level.unsqueeze(1) - unit * along.unsqueeze(1)) * d["rstd"].unsqueeze(1)
            return {"dx": dx + d["dsum"] if case["residual"] else dx, "dweight": torch.einsum("mc,mc->c", d["dy"], unit),
                    "dbias": torch.einsum("mc->c", d["dy"])}
        v = torch.add(d["x"], d["residual"]) if case["residual"] else d["x"]
        spread, mean = torch.var_mean(v, dim=1, correction=0)
        rstd = torch.pow(spread + EPS, -0.5)
        y = torch.einsum("mc,m,c->mc", v - mean.unsqueeze(1), rstd, w) + d["bias"]
        out = {"mean": mean, "rstd": rstd, "y": y}
        if case["residual"]:
            out["sum"] = v
        if case["out"] == "e4m3":
            top = torch.linalg.vector_norm(y, ord=math.inf, dim=1)
            out["scale"] = torch.where(top > 0, top / F8_MAX, 1.0)
            out["y"] = y / out["scale"].unsqueeze(1)
        return out
    if case["op"] == "dropout":
        lots = lots64(d["x"].numel(), s["seed"], s["offset"])
        least = int(np.rint(case["p"] * 65536))
        factor = torch.from_numpy((lots >= least) * (65536.0 / (65536 - least))).to(d["x"].device).reshape(d["x"].shape)
        return torch.addcmul(d["residual"], d["x"], factor) if case["residual"] else d["x"] * factor
    n, a = case["n"], case["smoothing"]
    z = torch.mm(d["x"], d["w"].t())
    if case["bias"]:
        z += d["bias"]
    counts = s["target"] != IGNORE
    # the distribution a row should have
    goal = torch.zeros_like(z)
    goal.scatter_(1, s["target"].clamp(min=0).unsqueeze(1), 1.0 - a)
    goal += a / n
    if case["backward"]:
        g = d["dloss"] * counts
        if case["reduction"] == "mean":
            g = g / counts.sum()
        z -= d["lse"].unsqueeze(1)
        dz = torch.mul(z.exp_() - goal, g.unsqueeze(1))
        out = {"dx": torch.mm(dz, d["w"]), "dw": torch.mm(dz.t(), d["x"])}
        if case["bias"]:
            out["dbias"] = torch.mv(dz.t(), torch.ones_like(dz[:, 0]))
        return out
    lse = torch.logsumexp(z, dim=1)
    each = (lse - torch.einsum("mn,mn->m", goal, z)) * counts
    if case["reduction"] == "mean":
        each = each.sum() / counts.sum()
    elif case["reduction"] == "sum":
        each = each.sum()
    return {"loss": each, "lse": lse}
