"""GPU parity of the feed-forward operators where the first suite's sizes do not reach: few rows (the kernels that keep a
weight row in one workgroup), whole tiles' epilogues, steep arguments and tiny scales, and the example that runs them
together.  Tolerances count roundings (feed_forward_ref)."""
import os
import sys

import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
from test_feed_forward_gpu import ACTS, BF16, E4M3, F32, dev, pitched, quantised, values

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 3, 16, 17, 31, 32, 33]
# one element; a piece; past whole turns of 256 and 2048 bytes and short of them; long rows; unaligned ones
WEIGHTS = [(1, 1), (17, 8), (33, 127), (200, 1000), (40, 2048), (24, 4099), (250, 9216)]


@pytest.mark.parametrize("n,k", WEIGHTS)
@pytest.mark.parametrize("dtype", [F32, BF16, E4M3])
def test_few_rows(n, k, dtype):
    out = F32 if dtype is F32 else BF16
    for m in ROWS:
        name = ACTS[(m + n) % 5]
        if dtype is E4M3:
            x, xs = quantised(1, m, k)
            (w, ws), (wu, us) = quantised(2, n, k, std=k ** -0.5), quantised(3, n, k, std=k ** -0.5)
        else:
            xs = ws = us = None
            x, w, wu = (values(s, *size, std=std, dtype=dtype) for s, size, std in
                        ((1, (m, k), 1.0), (2, (n, k), k ** -0.5), (3, (n, k), k ** -0.5)))
        bias, res = values(4, n, dtype=out), values(5, m, n, dtype=out)
        y, z = mic.linear(x, w, bias=bias, residual=res, activation=name, x_scale=xs, w_scale=ws, return_preact=True)
        ref_y, ref_z = R.linear(x, w, bias, res, name, out, xs, ws)
        R.check(z, ref_z, "preact %d %s" % (m, name))
        R.check(y, ref_y, "y %d %s" % (m, name))
        h, gate, up = mic.gated_linear(x, w, wu, activation=name, x_scale=xs, w_gate_scale=ws, w_up_scale=us,
                                       return_products=True)
        ref = R.gated(x, w, wu, name, out, xs, ws, us)
        for got, want, what in zip((h, gate, up), ref, ("h", "gate", "up")):
            R.check(got, want, "%s %d %s" % (what, m, name))


@pytest.mark.parametrize("m", [1, 2, 5, 20])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_rows_between_others(m, dtype):
    """Rows of a wider matrix, NaN beside them; one row that is no number reaches no other."""
    n, k = 40, 1101
    x, w, wu = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype), values(3, n, k, dtype=dtype)
    R.check(mic.linear(pitched(x, 3, 1), pitched(w, 5, 3)), R.linear(x, w, None, None, "none", dtype)[0], "padded")
    R.check(mic.gated_linear(pitched(x, 3, 1), pitched(w, 5, 3), pitched(wu, 2, 1)), R.gated(x, w, wu, "silu", dtype)[0],
            "padded gated")
    clean = mic.linear(x, w)
    x2, w2 = x.clone(), w.clone()
    x2[m - 1] = float("nan")
    w2[n - 1] = float("nan")
    y = mic.linear(x2, w2)
    assert torch.equal(y[: m - 1, : n - 1], clean[: m - 1, : n - 1])
    assert torch.isnan(y[m - 1]).all() and torch.isnan(y[:, n - 1]).all()


@pytest.mark.parametrize("m,n,k", [(512, 768, 640), (513, 1040, 264), (1000, 520, 1032)])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_whole_tile_epilogues(m, n, k, name):
    """Bias, scales, residual and preact together on tiles that are whole and tiles that are not, rows of each sampled."""
    g = torch.Generator().manual_seed(m)
    rows = torch.cat([torch.tensor([0, 31, 32, m - 1]), torch.randint(0, m, (40,), generator=g)]).to(dev())
    for dtype in (BF16, E4M3, F32):
        out = F32 if dtype is F32 else BF16
        xs = ws = None
        if dtype is E4M3:
            (x, xs), (w, ws) = quantised(1, m, k), quantised(2, n, k, std=k ** -0.5)
        else:
            x, w = values(1, m, k, dtype=dtype), values(2, n, k, std=k ** -0.5, dtype=dtype)
        bias, res = values(3, n, dtype=out), values(4, m, n, dtype=out)
        y, z = mic.linear(x, w, bias=bias, residual=res, activation=name, x_scale=xs, w_scale=ws, return_preact=True)
        ref_y, ref_z = R.linear(x[rows], w, bias, res[rows], name, out, None if xs is None else xs[rows], ws)
        R.check(y[rows], ref_y, "y %s" % dtype)
        R.check(z[rows], ref_z, "preact %s" % dtype)
        assert torch.equal(mic.linear(x, w, bias=bias, residual=res, activation=name, x_scale=xs, w_scale=ws), y)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steep_arguments(dtype):
    """Far from zero an activation is 0 or z and its slope 0 or 1, also where z^2 is past fp32's range."""
    z = torch.tensor([[-3e38, -1e20, -1e10, -200.0, 200.0, 1e10, 1e20, 3e38]], device=dev()).to(dtype)
    n = z.shape[1]
    eye = torch.eye(n, device=dev()).to(dtype)
    one = torch.ones_like(z)
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        want = z.clamp(min=0)
        assert torch.equal(mic.linear(z, eye, activation=name), want), name
        dx, _, db = mic.linear_backward(one, z, eye, preact=z, activation=name, bias=True)
        step = (z > 0).to(dtype)
        assert torch.equal(dx, step) and torch.equal(db, step[0]), name
    inf = torch.full((1, 1), float("inf"), device=dev()).to(dtype)
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        assert torch.equal(mic.linear(inf, eye[:1, :1], activation=name), inf), name


def test_norm_scales_below_the_normal_numbers():
    """A row whose scale's reciprocal overflows: y / scale all the same, zeros stay zeros."""
    x = values(1, 3, 96)
    x[:, 5] = 0
    w = torch.full((96,), 1e-37, device=dev())
    r = mic.rms_norm(x, w, eps=1e-6, out_dtype=E4M3)
    scale = r.scale.double()
    assert (scale > 0).all() and (scale < 2.0 ** -126).all()
    s = x.double()
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * w.double()
    got = r.y.double()
    assert not got[:, 5].any() and torch.isfinite(got).all()
    # y and the scale are multiples of 2^-149, y / scale rounds to e4m3: half a step, or half of the smallest number
    v = y / scale[:, None]
    bound = 2.0 ** -4 * v.abs() + 2.0 ** -10 + (0.5 * 2.0 ** -149 / scale)[:, None] * 2 + 1e-4 * v.abs()
    assert ((got - v).abs() <= bound).all()
    top = y.abs().amax(1) / 448.0
    assert ((scale - top).abs() <= 2.0 ** -149 + 1e-5 * top).all()


def test_many_partial_sums():
    """Column sums joined from more groups than a block has lanes of rows."""
    m, n = 5000, 72
    for dtype in (F32, BF16):
        dy, s, w = values(1, m, n, dtype=dtype), values(2, m, n, dtype=dtype), values(3, n, dtype=dtype)
        rstd = (s.float().square().mean(1) + 1e-6).rsqrt()
        dx, dw = mic.rms_norm_backward(dy, s, w, rstd)
        ref = R.rms_norm_backward(dy, s, w, rstd, None)
        R.check(dx, ref[0], "dx")
        R.check(dw, ref[1], "dweight")
        db = mic.linear_backward(dy, s[:, :8].contiguous(), values(4, n, 8, dtype=dtype), bias=True)[2]
        R.check(db, R.linear_backward(dy, s[:, :8], values(4, n, 8, dtype=dtype), None, "none")[2], "dbias")


def test_example_trains_and_serves():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import feed_forward
    finally:
        sys.path.pop(0)
    losses, error, token_error = feed_forward.main(["--width", "256", "--hidden", "520", "--tokens", "512", "--steps", "30"])
    assert losses[-1] < 0.8 * losses[0]
    # each of the two quantised operands is off by at most 2^-4 of an element, most by far less, at random
    assert error < 0.1 and token_error < 0.15


class _Declines:
    """Stands for the native binding where it takes no argument list."""

    def __getattr__(self, name):
        return lambda *args: None


def test_both_ways_into_the_library_agree(monkeypatch):
    from convolution_forward_conv2d_amd import feed_forward as F
    m, n, k = 37, 136, 264

    def results():
        out = []
        for dtype in (F32, BF16):
            x, w, wu = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype), values(3, n, k, dtype=dtype)
            bias, res, weight, s = (values(4, n, dtype=dtype), values(5, m, n, dtype=dtype), values(6, k, dtype=dtype),
                                    values(7, m, k, dtype=dtype))
            for r in (mic.rms_norm(x, weight), mic.rms_norm(x, weight, residual=s, out_dtype=E4M3, eps=1e-5)):
                out += list(r)
                out += list(mic.rms_norm_backward(s, r.sum, weight, r.rstd))
            out += list(mic.rms_norm_backward(s, x, weight, r.rstd, dsum=x))
            y, z = mic.linear(x, w, bias=bias, residual=res, activation="gelu", return_preact=True)
            out += [y, z, mic.linear(x, w), mic.linear(x.reshape(1, m, k), w)]
            out += list(mic.linear_backward(res, x, w, preact=z, activation="gelu", bias=True))
            out += list(mic.linear_backward(res, x, w))
            h, gate, up = mic.gated_linear(x, w, wu, return_products=True, activation="relu")
            out += [h, gate, up, mic.gated_linear(x, w, wu)]
            out += list(mic.gated_linear_backward(res, x, w, wu, gate, up))
        (x, xs), (w, ws), (wu, us) = quantised(1, m, k), quantised(2, n, k), quantised(3, n, k)
        for o in (None, BF16, F32):
            for fast in (False, True):
                out.append(mic.linear(x, w, x_scale=xs, w_scale=ws, out_dtype=o, fast_sums=fast))
                out.append(mic.gated_linear(x, w, wu, x_scale=xs, w_gate_scale=ws, w_up_scale=us, out_dtype=o, fast_sums=fast))
        return out

    native = results()
    monkeypatch.setattr(F, "_native", _Declines())
    general = results()
    assert len(native) == len(general)
    for a, b in zip(native, general):
        assert (a is None) == (b is None)
        if a is not None:
            assert a.dtype is b.dtype and a.shape == b.shape
            as_bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
            assert torch.equal(a.view(as_bits), b.view(as_bits))


def test_refusals_name_the_argument():
    """Arguments the native binding declines are refused by the checks behind it."""
    x, w, b = values(1, 4, 8), values(2, 3, 8), values(3, 3)
    for call, error, match in (
            (lambda: mic.linear(x, w.to(BF16)), TypeError, "w must be"),
            (lambda: mic.linear(x, w[:, :7]), ValueError, "w has shape"),
            (lambda: mic.linear(x, w.cpu()), ValueError, "w is on"),
            (lambda: mic.linear(x, w, bias=b[:2]), ValueError, "bias"),
            (lambda: mic.linear(x, w, residual=x), ValueError, "residual"),
            (lambda: mic.linear(x, w, activation="swish"), ValueError, "activation"),
            (lambda: mic.linear(x, w, out_dtype=BF16), TypeError, "out_dtype"),
            (lambda: mic.linear(x, w, x_scale=b, w_scale=b), ValueError, "scales"),
            (lambda: mic.linear(x.to(E4M3), w.to(E4M3)), ValueError, "scales"),
            (lambda: mic.linear_backward(b.expand(4, 3).contiguous(), x, w, activation="relu"), ValueError, "preact"),
            (lambda: mic.gated_linear(x, w, w[:2]), ValueError, "output features"),
            (lambda: mic.gated_linear_backward(b.expand(4, 3).contiguous(), x, w, w, x, x), ValueError, "gate"),
            (lambda: mic.rms_norm(x, b), ValueError, "weight"),
            (lambda: mic.rms_norm(x, w[0], residual=x[:2]), ValueError, "residual"),
            (lambda: mic.rms_norm(x, w[0], eps=-1.0), ValueError, "eps"),
            (lambda: mic.rms_norm(x, w[0], out_dtype=BF16), TypeError, "out_dtype"),
            (lambda: mic.rms_norm_backward(x, x, w[0], b), ValueError, "rstd")):
        with pytest.raises(error, match=match):
            call()
