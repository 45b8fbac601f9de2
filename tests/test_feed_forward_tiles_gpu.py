"""GPU parity of every kernel that the feed-forward products take, each named, on sizes with remainders.

Every element of every output is compared with 64 bits, within bounds that count roundings (feed_forward_ref, whose sums
run on the GPU here).  A second call finds the same operands between NaN, at the same alignment, and has to give the same
bits.
"""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
from feed_forward_tiles import cases, planned, product_of
from test_feed_forward_gpu import BF16, E4M3, F32, dev, pitched

pytestmark = pytest.mark.gpu

CASES = list(cases())
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
TYPES = {"f32": F32, "bf16": BF16, "e4m3": E4M3}


@pytest.fixture(autouse=True)
def sums_on_the_gpu(monkeypatch):
    monkeypatch.setattr(R, "d", lambda t: None if t is None else t.detach().to(dev()).double())


def maker(seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return lambda *shape, std=1.0, dtype=F32: torch.randn(shape, generator=g, device=dev()).mul_(std).to(dtype)


def rows_quantised(v):
    scale = v.abs().amax(1) / 448.0
    return (v / scale[:, None]).clamp(-448, 448).to(E4M3), scale


def forward(op, dtype, fast, m, n, k, aligned, act):
    values = maker(m + n + k)
    wide = {"f32": F32, "bf16": BF16}.get(dtype)
    scales = {}
    if dtype == "e4m3":
        x, xs = rows_quantised(values(m, k))
        (w, ws), (u, us) = (rows_quantised(values(n, k, std=k ** -0.5)) for _ in range(2))

        def short(scale, v):       # of 64 products added by the e4m3 instruction, 2^-11 of the largest
            if not fast:
                return 0.0
            top = (R.d(x).abs().amax(1) * R.d(xs))[:, None] * (R.d(v).abs().amax(1) * R.d(scale))
            return 1.01 * -(-k // 64) * 2.0 ** -11 * top
    else:
        x, xs, w, ws, u, us = (values(m, k, dtype=wide), None, values(n, k, std=k ** -0.5, dtype=wide), None,
                               values(n, k, std=k ** -0.5, dtype=wide), None)
        short = lambda scale, v: 0.0
    pad = 16 // x.element_size() if aligned else 3
    x2, w2, u2 = (pitched(t, pad, 0 if aligned else 1) for t in (x, w, u))
    for out in ((BF16, F32) if dtype == "e4m3" else (wide,)):
        if op == "linear":
            bias, res = values(n, dtype=out), values(m, n, dtype=out)
            # the bound of fast sums passes the activations that have no kink and slope at most 1.13
            name = act if not fast else "none"
            y, z = mic.linear(x, w, bias, res, name, xs, ws, out, return_preact=True, fast_sums=fast)
            ref_y, ref_z = R.linear(x, w, bias, res, name, out, xs, ws)
            R.check(z, (ref_z[0], ref_z[1] + short(ws, w)), "preact")
            R.check(y, (ref_y[0], ref_y[1] + short(ws, w)), "y")
            assert torch.equal(y, mic.linear(x2, w2, bias, res, name, xs, ws, out, fast_sums=fast))
            assert torch.equal(z, mic.linear(x, w, bias, None, "none", xs, ws, out, fast_sums=fast))
        else:
            name = act if not fast else "none"
            h, gate, up = mic.gated_linear(x, w, u, name, xs, ws, us, out, return_products=True, fast_sums=fast)
            ref_h, ref_g, ref_u = R.gated(x, w, u, name, out, xs, ws, us)
            eg, eu = short(ws, w), short(us, u)
            R.check(gate, (ref_g[0], ref_g[1] + eg), "gate")
            R.check(up, (ref_u[0], ref_u[1] + eu), "up")
            R.check(h, (ref_h[0], ref_h[1] + eg * ref_u[0].abs() + eu * ref_g[0].abs() + eg * eu), "h")
            assert torch.equal(h, mic.gated_linear(x2, w2, u2, name, xs, ws, us, out, fast_sums=fast))


def backward(op, dtype, m, n, k, aligned, act):
    values = maker(m + n + k)
    t = TYPES[dtype]
    dy, x, z = values(m, n, dtype=t), values(m, k, dtype=t), values(m, n, dtype=t)
    w = values(n, k, std=n ** -0.5, dtype=t)
    pad, offset = (16 // x.element_size(), 0) if aligned else (3, 1)

    def put(v):
        return pitched(v, pad, offset)
    if op == "gb":
        u, wu = values(m, n, dtype=t), values(n, k, std=n ** -0.5, dtype=t)
        got = mic.gated_linear_backward(dy, x, w, wu, z, u, act)
        again = mic.gated_linear_backward(put(dy), put(x), put(w), put(wu), put(z), put(u), act)
        ref, what = R.gated_backward(dy, x, w, wu, z, u, act), ("dx", "dw_gate", "dw_up")
    else:
        got = mic.linear_backward(dy, x, w, z, act, bias=True)
        again = mic.linear_backward(put(dy), put(x), put(w), put(z), act, bias=True)
        ref, what = R.linear_backward(dy, x, w, z, act), ("dx", "dw", "dbias")
    for g, a, want, name in zip(got, again, ref, what):
        R.check(g, want, name)
        assert torch.equal(g, a), name


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_a_kernel(case):
    _, op, dtype, fast, m, n, k, aligned, name = case
    # the plan of the card at hand: whole, unless it is partitioned
    assert torch.cuda.get_device_properties(dev()).multi_processor_count == 256
    assert product_of(op, name, planned(op, dtype, fast, m, n, k, aligned)) == name
    act = "none" if op == "l0" else ACTS[1 + (m + n + k) % 4]
    if op in ("linear", "gated"):
        forward(op, dtype, fast, m, n, k, aligned, act)
    else:
        backward(op, dtype, m, n, k, aligned, act)
