"""The feed-forward operators as they are used: cases, inputs, plain forms and 64-bit results.

Three operators and their gradients, in the order a feed-forward sublayer runs them:

  norm       s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight, y in x's type or in e4m3 with a scale per row
  gated      h = act(x Wg^T) * (x Wu^T)
  linear     y = act(x W^T + bias) + residual

``run`` computes a case either with the library's entry points (``own``) or in plain torch, in 32 bits.
"""
import math

import torch

own = False

EPS = 1e-6
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": F8}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1}

# The widths are the library's own fully-connected ones: 4096 features, 9216 = 256 x 6 x 6 in the wide layer, 1000 classes.


def listed():
    return [
        # the norm of one token between two layers while serving: launch latency
        norm("norm_token", 1, 4096, "bf16", "bf16", True),
        # a long prompt's norm, quantised by rows for an 8-bit product; odd row count
        norm("norm_prompt_e4m3", 2047, 4096, "bf16", "e4m3", True),
        # a training step's norm gradient
        norm("norm_train_backward", 8192, 4096, "bf16", "bf16", True, backward=True),
        # the projection back of one token while serving: weights stream once from memory
        linear("linear_token", 1, 4096, 9216, "bf16", "none", False, True),
        # AlexNet's fc6 in its own type, with the bias and ReLU the network has there
        linear("linear_fc6_f32", 128, 4096, 9216, "f32", "relu", True, False),
        # a classifier head where nothing is a multiple of anything: rows, outputs and features odd, rows unaligned
        linear("linear_odd", 131, 1001, 4093, "bf16", "none", True, False),
        # the projection back of a long prompt or a training batch, with the residual
        linear("linear_rows", 8192, 4096, 9216, "bf16", "none", False, True),
        # 8-bit serving: rows and weights in e4m3 with scales
        linear("linear_rows_e4m3", 4096, 9216, 4096, "e4m3", "gelu", True, False),
        # a training step's gradients of a layer with bias and GELU
        linear("linear_train_backward", 4096, 4096, 9216, "bf16", "gelu", True, False, backward=True),
        # four sequences' next tokens through the gated projections
        gated("gated_tokens", 4, 9216, 4096, "bf16", "silu"),
        # a prompt's gated projections
        gated("gated_rows", 4096, 9216, 4096, "bf16", "silu"),
        # their gradients in a training step
        gated("gated_train_backward", 4096, 9216, 4096, "bf16", "silu", backward=True),
    ]


def norm(name, m, c, dtype, out, residual, backward=False):
    return {"name": name, "op": "norm", "m": m, "c": c, "dtype": dtype, "out": out, "residual": residual,
            "backward": backward}


def linear(name, m, n, k, dtype, act, bias, residual, backward=False):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "backward": backward}


def gated(name, m, n, k, dtype, act, backward=False):
    return {"name": name, "op": "gated", "m": m, "n": n, "k": k, "dtype": dtype, "act": act, "backward": backward}


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        kind = rng.random()          # mostly whole tiles' multiples, as layers have; odd ones among them
        if kind < 0.4 and v >= 64:
            v -= v % 64
        elif kind < 0.7 and v >= 8:
            v -= v % 8
        return v

    op = rng.choice(["norm", "linear", "gated"])
    backward = rng.random() < 0.4
    m = size(64 if backward else 1, 8192)
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        out = dtype if backward or rng.random() < 0.5 else "e4m3"
        case = norm("", m, size(256, 9216), dtype, out, rng.random() < 0.7, backward)
    else:
        n, k = size(256, 9216), size(256, 9216)
        dtype = rng.choice(["bf16", "bf16", "f32"] if backward else ["bf16", "bf16", "f32", "e4m3"])
        act = rng.choice(["relu", "gelu", "gelu_tanh", "silu"] + (["none"] if op == "linear" else []))
        most = (1 << 37) if op == "linear" else (1 << 36)
        m = max(1, min(m, most // (n * k)))
        if op == "linear":
            case = linear("", m, n, k, dtype, act, rng.random() < 0.5, not backward and rng.random() < 0.5, backward)
        else:
            case = gated("", m, n, k, dtype, act, backward)
    del case["name"]
    return case


def work(case):
    m, e = case["m"], BYTES[case["dtype"]]
    if case["op"] == "norm":
        c = case["c"]
        if case["backward"]:         # dy, s and the gradient that reaches s directly in, ds out; weight, its gradient and 1/rms
            return {"bytes": m * c * e * (4 if case["residual"] else 3) + 2 * c * e + 4 * m, "flops": 10.0 * m * c}
        one = m * c * e
        return {"bytes": one * (3 if case["residual"] else 1) + m * c * BYTES[case["out"]] + c * e + 8 * m,
                "flops": 6.0 * m * c}
    n, k = case["n"], case["k"]
    two = 2 if case["op"] == "gated" else 1
    if case["backward"]:             # dy, x, W and the saved products in; dx and dW out
        return {"bytes": e * (m * n * (1 + (two if case["act"] != "none" or two == 2 else 0)) + 2 * m * k + 2 * two * n * k)
                + (n * e if case.get("bias") else 0),
                "flops": 4.0 * two * m * n * k}
    o = BYTES[out_type(case)]
    scales = 4 * (m + two * n) if case["dtype"] == "e4m3" else 0
    return {"bytes": e * (m * k + two * n * k) + o * m * n * (2 if case.get("residual") else 1)
            + (n * o if case.get("bias") else 0) + scales,
            "flops": 2.0 * two * m * n * k}


def out_type(case):
    return "bf16" if case["dtype"] == "e4m3" else case["dtype"]


# ---------------------------------------------------------------- inputs


def quantise_rows(v):
    """Rows in e4m3 and their scales, as a user's weights or activations are kept."""
    scale = v.abs().amax(dim=1) / F8_MAX
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (v / scale[:, None]).clamp(-F8_MAX, F8_MAX).to(F8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=None):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype or dt)

    m = case["m"]
    s = {"case": dict(case)}
    if case["op"] == "norm":
        c = case["c"]
        s["weight"] = normal(c, std=0.1, dtype=torch.float32).add_(1.0).to(dt)
        if case["backward"]:
            s["sum"] = normal(m, c, std=1.5)
            s["rstd"] = (s["sum"].float().square().mean(dim=1) + EPS).rsqrt()
            s["dy"] = normal(m, c, std=0.5)
            s["dsum"] = normal(m, c, std=0.5) if case["residual"] else None
        else:
            s["x"] = normal(m, c)
            s["residual"] = normal(m, c, std=2.0) if case["residual"] else None
        return s
    n, k = case["n"], case["k"]
    names = ["w_gate", "w_up"] if case["op"] == "gated" else ["w"]
    if case["dtype"] == "e4m3":
        s["x"], s["x_scale"] = quantise_rows(normal(m, k, dtype=torch.float32))
        for w in names:
            s[w], s[w + "_scale"] = quantise_rows(normal(n, k, std=k ** -0.5, dtype=torch.float32))
    else:
        s["x"] = normal(m, k)
        s["x_scale"] = None
        for w in names:
            s[w], s[w + "_scale"] = normal(n, k, std=k ** -0.5), None
    o = TYPES[out_type(case)]
    if case["backward"]:
        s["dy"] = normal(m, n)
        # what the forward pass kept for its gradient
        if case["op"] == "gated":
            s["gate"] = (s["x"].float() @ s["w_gate"].float().t()).to(o)
            s["up"] = (s["x"].float() @ s["w_up"].float().t()).to(o)
        elif case["act"] != "none":
            s["preact"] = (s["x"].float() @ s["w"].float().t() + 0.1).to(o)
        else:
            s["preact"] = None
    elif case["op"] == "linear":
        s["bias"] = normal(n, std=0.1, dtype=o) if case["bias"] else None
        s["residual"] = normal(m, n, dtype=o) if case["residual"] else None
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(s):
    import convolution_forward_conv2d_amd as mic

    case = s["case"]
    if case["op"] == "norm":
        if case["backward"]:
            dx, dweight = mic.rms_norm_backward(s["dy"], s["sum"], s["weight"], s["rstd"], dsum=s["dsum"])
            return {"dx": dx, "dweight": dweight}
        r = mic.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out_dtype=TYPES[case["out"]])
        out = {"y": r.y, "rstd": r.rstd}
        if case["residual"]:
            out["sum"] = r.sum
        if case["out"] == "e4m3":
            out["scale"] = r.scale
        return out
    if case["op"] == "linear":
        if case["backward"]:
            dx, dw, dbias = mic.linear_backward(s["dy"], s["x"], s["w"], preact=s["preact"], activation=case["act"],
                                                bias=case["bias"])
            return {"dx": dx, "dw": dw, "dbias": dbias} if case["bias"] else {"dx": dx, "dw": dw}
        # fast_sums concerns the e4m3 cases: a user who takes that type serves, and asks for its rate
        return mic.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], activation=case["act"],
                          x_scale=s["x_scale"], w_scale=s["w_scale"], out_dtype=TYPES[out_type(case)], fast_sums=True)
    if case["backward"]:
        dx, dwg, dwu = mic.gated_linear_backward(s["dy"], s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"],
                                                 activation=case["act"])
        return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}
    return mic.gated_linear(s["x"], s["w_gate"], s["w_up"], activation=case["act"], x_scale=s["x_scale"],
                            w_gate_scale=s["w_gate_scale"], w_up_scale=s["w_up_scale"],
                            out_dtype=TYPES[out_type(case)], fast_sums=True)


def activate(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def slope(z, act):
    """d activate / d z."""
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def product(x, w, x_scale, w_scale):
    z = x.float() @ w.float().t()
    if x_scale is not None:
        z = z * x_scale[:, None] * w_scale[None, :]
    return z


def run_plain(s):
    case = s["case"]
    dt = TYPES[case["dtype"]]
    if case["op"] == "norm":
        w = s["weight"].float()
        if case["backward"]:
            v, dy, rstd = s["sum"].float(), s["dy"].float(), s["rstd"][:, None]
            wdy = w * dy
            ds = rstd * (wdy - v * rstd * rstd * (wdy * v).mean(dim=1, keepdim=True))
            if case["residual"]:
                ds = ds + s["dsum"].float()
            return {"dx": ds.to(dt), "dweight": (dy * v * rstd).sum(dim=0).to(dt)}
        v = s["x"].float()
        if case["residual"]:
            v = v + s["residual"].float()
        rstd = 1 / torch.sqrt((v * v).mean(dim=1) + EPS)
        y = v * rstd[:, None] * w
        out = {"rstd": rstd}
        if case["residual"]:
            out["sum"] = v.to(dt)
        if case["out"] == "e4m3":
            out["y"], out["scale"] = quantise_rows(y)
        else:
            out["y"] = y.to(dt)
        return out
    o = TYPES[out_type(case)]
    if case["op"] == "linear":
        if case["backward"]:
            dz = s["dy"].float()
            if case["act"] != "none":
                dz = dz * slope(s["preact"].float(), case["act"])
            out = {"dx": (dz @ s["w"].float()).to(o), "dw": (dz.t() @ s["x"].float()).to(o)}
            if case["bias"]:
                out["dbias"] = dz.sum(dim=0).to(o)
            return out
        z = product(s["x"], s["w"], s["x_scale"], s["w_scale"])
        if case["bias"]:
            z = z + s["bias"].float()
        y = activate(z, case["act"])
        if case["residual"]:
            y = y + s["residual"].float()
        return y.to(o)
    if case["backward"]:
        gate, up, dh, x = s["gate"].float(), s["up"].float(), s["dy"].float(), s["x"].float()
        dg = dh * up * slope(gate, case["act"])
        du = dh * activate(gate, case["act"])
        return {"dx": (dg @ s["w_gate"].float() + du @ s["w_up"].float()).to(o), "dw_gate": (dg.t() @ x).to(o),
                "dw_up": (du.t() @ x).to(o)}
    gate = product(s["x"], s["w_gate"], s["x_scale"], s["w_gate_scale"])
    up = product(s["x"], s["w_up"], s["x_scale"], s["w_up_scale"])
    return (activate(gate, case["act"]) * up).to(o)


# ---------------------------------------------------------------- the definition in 64 bits


def act64(z, act):
    """(value, derivative) at z, from the distribution functions the activations are defined by."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = (z > 0).double()
        return on * z, on
    if act == "gelu":                # z times the normal distribution function
        phi = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":           # the logistic function of twice tanh's argument
        a = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(a * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * a * (1 + 0.134145 * z ** 2)
    p = torch.sigmoid(z)
    return z * p, p + z * p * (1 - p)


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    if case["op"] == "norm":
        w = d["weight"]
        if case["backward"]:
            unit = d["sum"] * d["rstd"].unsqueeze(1)
            along = torch.einsum("mc,c,mc->m", d["dy"], w, unit) / case["c"]
            dx = (d["dy"] * w - unit * along.unsqueeze(1)) * d["rstd"].unsqueeze(1)
            return {"dx": dx + d["dsum"] if case["residual"] else dx, "dweight": torch.einsum("mc,mc->c", d["dy"], unit)}
        v = torch.add(d["x"], d["residual"]) if case["residual"] else d["x"]
        rstd = torch.pow(torch.linalg.vector_norm(v, dim=1).square() / case["c"] + EPS, -0.5)
        y = torch.einsum("mc,m,c->mc", v, rstd, w)
        out = {"rstd": rstd, "y": y}
        if case["residual"]:
            out["sum"] = v
        if case["out"] == "e4m3":
            top = torch.linalg.vector_norm(y, ord=math.inf, dim=1)
            out["scale"] = torch.where(top > 0, top / F8_MAX, 1.0)
            out["y"] = y / out["scale"].unsqueeze(1)
        return out
    for name in ("x", "w", "w_gate", "w_up"):
        if name + "_scale" in d:
            d[name] = torch.einsum("ij,i->ij", d[name], d[name + "_scale"])
    if case["op"] == "linear":
        if case["backward"]:
            dz = d["dy"] if case["act"] == "none" else d["dy"] * act64(d["preact"], case["act"])[1]
            out = {"dx": torch.mm(dz, d["w"]), "dw": torch.mm(dz.t(), d["x"])}
            if case["bias"]:
                out["dbias"] = torch.mv(dz.t(), torch.ones_like(dz[:, 0]))
            return out
        z = torch.mm(d["x"], d["w"].t())
        if case["bias"]:
            z += d["bias"]
        y = act64(z, case["act"])[0]
        return y + d["residual"] if case["residual"] else y
    if case["backward"]:
        value, rise = act64(d["gate"], case["act"])
        d_both = torch.cat([d["dy"] * d["up"] * rise, d["dy"] * value], dim=1)
        d_w = torch.mm(d_both.t(), d["x"])
        return {"dx": torch.mm(d_both, torch.cat([d["w_gate"], d["w_up"]])), "dw_gate": d_w[: case["n"]],
                "dw_up": d_w[case["n"]:]}
    return act64(torch.mm(d["x"], d["w_gate"].t()), case["act"])[0] * torch.mm(d["x"], d["w_up"].t())
