"""GPU parity of the feed-forward operators against plain 64-bit forms.

Each case's tolerance comes from counting its roundings (feed_forward_ref).
Sizes sit where kernels can go wrong: one row, one feature, one past and one
short of every tile, unaligned rows, padded pitches, split reductions.
"""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def dev():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    return torch.device("cuda", 0)


def values(seed, *shape, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(dev())


def pitched(t, pad, offset=0):
    """t's values in rows `pad` elements further apart, `offset` elements into an allocation, NaN around them."""
    m, n = t.shape
    base = torch.full((offset + m * (n + pad) + 1,), float("nan"), dtype=torch.float32, device=t.device).to(t.dtype)
    v = base.as_strided((m, n), (n + pad, 1), offset)
    v.copy_(t)
    return v


def quantised(seed, m, k, std=1.0):
    v = values(seed, m, k, std=std)
    scale = v.abs().amax(1) / 448.0 if k else torch.ones(m, device=dev())
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (v / scale[:, None]).clamp(-448, 448).to(E4M3), scale


SIZES = [(1, 1, 1), (1, 17, 8), (1, 200, 1000), (2, 64, 64), (3, 33, 31), (5, 40, 136), (16, 256, 512), (17, 130, 96),
         (31, 65, 257), (33, 127, 129), (64, 64, 64), (65, 63, 65), (100, 72, 1000), (128, 128, 128), (129, 257, 63),
         (200, 264, 328), (257, 129, 520), (300, 96, 2049), (256, 512, 256), (513, 384, 192), (640, 520, 264)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, E4M3])
def test_linear(m, n, k, dtype):
    pick = (m + n + k) % 5
    out = BF16 if dtype is not F32 and (m + k) % 3 else F32
    if dtype is BF16:
        out = BF16
    if dtype is E4M3:
        x, xs = quantised(1, m, k)
        w, ws = quantised(2, n, k, std=k ** -0.5)
    else:
        x, xs, w, ws = values(1, m, k, dtype=dtype), None, values(2, n, k, std=k ** -0.5, dtype=dtype), None
    for name, with_bias, with_residual in ((ACTS[pick], True, False), (ACTS[(pick + 1) % 5], False, True),
                                           (ACTS[(pick + 2) % 5], True, True)):
        bias = values(3, n, dtype=out) if with_bias else None
        res = values(4, m, n, dtype=out) if with_residual else None
        y, z = mic.linear(x, w, bias=bias, residual=res, activation=name, x_scale=xs, w_scale=ws, out_dtype=out,
                          return_preact=True)
        assert y.dtype is out and y.shape == (m, n) and z.shape == (m, n)
        ref_y, ref_z = R.linear(x, w, bias, res, name, out, xs, ws)
        R.check(z, ref_z, "preact %s" % name)
        R.check(y, ref_y, "y %s" % name)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, E4M3])
def test_gated(m, n, k, dtype):
    name = ACTS[(m + 2 * n + k) % 5]
    out = F32 if dtype is F32 else BF16
    if dtype is E4M3:
        x, xs = quantised(1, m, k)
        (wg, gs), (wu, us) = quantised(2, n, k, std=k ** -0.5), quantised(3, n, k, std=k ** -0.5)
    else:
        xs = gs = us = None
        x = values(1, m, k, dtype=dtype)
        wg, wu = (values(s, n, k, std=k ** -0.5, dtype=dtype) for s in (2, 3))
    h, gate, up = mic.gated_linear(x, wg, wu, activation=name, x_scale=xs, w_gate_scale=gs, w_up_scale=us,
                                   return_products=True)
    ref = R.gated(x, wg, wu, name, out, xs, gs, us)
    for got, want, what in zip((gate, up, h), (ref[1], ref[2], ref[0]), ("gate", "up", "h")):
        R.check(got, want, "%s %s" % (what, name))
    assert torch.equal(h, mic.gated_linear(x, wg, wu, activation=name, x_scale=xs, w_gate_scale=gs, w_up_scale=us))


@pytest.mark.parametrize("m,n,k", SIZES)
def test_fast_sums(m, n, k):
    """The e4m3 instruction: each of a sum's ceil(k / 64) groups is off by at most 2^-11 of its largest product, so
    by 2^-11 of max|x row| max|w row| at most, on top of the fp32 sum's own bound."""
    x, xs = quantised(1, m, k)
    (w, ws), (wu, us) = quantised(2, n, k, std=k ** -0.5), quantised(3, n, k, std=k ** -0.5)

    def short(v, scale):
        top = (R.d(x) * R.d(xs)[:, None]).abs().amax(1)[:, None] * (R.d(v) * R.d(scale)[:, None]).abs().amax(1)
        return -(-k // 64) * 2.0 ** -11 * top

    z = mic.linear(x, w, x_scale=xs, w_scale=ws, out_dtype=F32, fast_sums=True)
    value, bound = R.linear(x, w, None, None, "none", F32, xs, ws)[0]
    R.check(z, (value, bound + short(w, ws)), "z")
    h, gate, up = mic.gated_linear(x, w, wu, x_scale=xs, w_gate_scale=ws, w_up_scale=us, activation="relu",
                                   return_products=True, fast_sums=True)
    ref = R.gated(x, w, wu, "relu", BF16, xs, ws, us)
    R.check(gate, (ref[1][0], ref[1][1] + short(w, ws) * 1.01), "gate")
    R.check(up, (ref[2][0], ref[2][1] + short(wu, us) * 1.01), "up")
    eg, eu = short(w, ws), short(wu, us)
    R.check(h, (ref[0][0], ref[0][1] + 1.01 * (eg * ref[2][0].abs() + eu * ref[1][0].abs() + eg * eu)), "h")


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_linear_backward(m, n, k, dtype):
    for name, bias in ((ACTS[(m + n) % 5], True), (ACTS[(m + n + 2) % 5], False)):
        dy, x = values(1, m, n, dtype=dtype), values(2, m, k, dtype=dtype)
        w, z = values(3, n, k, std=n ** -0.5, dtype=dtype), values(4, m, n, dtype=dtype)
        dx, dw, db = mic.linear_backward(dy, x, w, preact=z, activation=name, bias=bias)
        ref = R.linear_backward(dy, x, w, z, name)
        R.check(dx, ref[0], "dx %s" % name)
        R.check(dw, ref[1], "dw %s" % name)
        if bias:
            R.check(db, ref[2], "dbias %s" % name)
        else:
            assert db is None


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_backward(m, n, k, dtype):
    name = ACTS[(m + n) % 5]
    dy, x = values(1, m, n, dtype=dtype), values(2, m, k, dtype=dtype)
    wg, wu = (values(s, n, k, std=n ** -0.5, dtype=dtype) for s in (3, 4))
    gate, up = (values(s, m, n, dtype=dtype) for s in (5, 6))
    got = mic.gated_linear_backward(dy, x, wg, wu, gate, up, activation=name)
    for g, want, what in zip(got, R.gated_backward(dy, x, wg, wu, gate, up, name), ("dx", "dw_gate", "dw_up")):
        R.check(g, want, "%s %s" % (what, name))


# past one tile of every shape, reductions of one, few and many steps, aligned rows and not
LARGE = [(256, 4096, 64), (512, 2048, 136), (1031, 1544, 264), (777, 2056, 520), (2048, 1100, 1032), (1500, 1501, 333),
         (300, 4100, 2056)]


@pytest.mark.parametrize("m,n,k", LARGE)
def test_large_products(m, n, k):
    """Every product of bf16 and e4m3 on the large tiles; sampled rows and columns against 64 bits."""
    g = torch.Generator().manual_seed(m + n + k)
    rows = torch.cat([torch.tensor([0, m - 1]), torch.randint(0, m, (30,), generator=g)]).to(dev())
    cols = torch.cat([torch.tensor([0, n - 1]), torch.randint(0, n, (30,), generator=g)]).to(dev())
    kcols = torch.cat([torch.tensor([0, k - 1]), torch.randint(0, k, (30,), generator=g)]).to(dev())

    def at(t, r, c):
        return t[r][:, c]

    x, w, wu = values(1, m, k, dtype=BF16), values(2, n, k, std=k ** -0.5, dtype=BF16), \
        values(3, n, k, std=k ** -0.5, dtype=BF16)
    bias, res = values(4, n, dtype=BF16), values(5, m, n, dtype=BF16)
    y, z = mic.linear(x, w, bias=bias, residual=res, activation="gelu", return_preact=True)
    ref = R.linear(x[rows], w[cols], bias[cols], at(res, rows, cols), "gelu", BF16)
    R.check(at(y, rows, cols), ref[0], "y")
    R.check(at(z, rows, cols), ref[1], "preact")
    h, gate, up = mic.gated_linear(x, w, wu, return_products=True)
    ref = R.gated(x[rows], w[cols], wu[cols], "silu", BF16)
    for got, want, what in zip((h, gate, up), ref, ("h", "gate", "up")):
        R.check(at(got, rows, cols), want, what)

    dy, wb, wub = res, w * k ** 0.5, wu * k ** 0.5
    dx, dw, db = mic.linear_backward(dy, x, wb, preact=z, activation="gelu", bias=True)
    R.check(at(dx, rows, kcols), R.linear_backward(dy[rows], x[rows], wb[:, kcols], z[rows], "gelu")[0], "dx")
    ref = R.linear_backward(dy[:, cols], x[:, kcols], wb[cols][:, kcols], z[:, cols], "gelu")
    R.check(at(dw, cols, kcols), ref[1], "dw")
    R.check(db[cols], ref[2], "dbias")
    dx, dw, _ = mic.linear_backward(dy, x, wb)
    R.check(at(dx, rows, kcols), R.linear_backward(dy[rows], x[rows], wb[:, kcols], None, "none")[0], "dx, dz = dy")
    R.check(at(dw, cols, kcols), R.linear_backward(dy[:, cols], x[:, kcols], wb[cols][:, kcols], None, "none")[1],
            "dw, dz = dy")
    dx, dg, du = mic.gated_linear_backward(dy, x, wb, wub, gate, up)
    R.check(at(dx, rows, kcols), R.gated_backward(dy[rows], x[rows], wb[:, kcols], wub[:, kcols], gate[rows], up[rows],
                                                  "silu")[0], "gated dx")
    ref = R.gated_backward(dy[:, cols], x[:, kcols], wb[cols][:, kcols], wub[cols][:, kcols], gate[:, cols],
                           up[:, cols], "silu")
    R.check(at(dg, cols, kcols), ref[1], "dw_gate")
    R.check(at(du, cols, kcols), ref[2], "dw_up")

    (x8, xs), (w8, ws), (u8, us) = quantised(6, m, k), quantised(7, n, k, std=k ** -0.5), quantised(8, n, k, std=k ** -0.5)
    for fast in (False, True):
        def short(v, scale):
            top = (R.d(x8[rows]) * R.d(xs[rows])[:, None]).abs().amax(1)[:, None] \
                * (R.d(v[cols]) * R.d(scale[cols])[:, None]).abs().amax(1)
            return -(-k // 64) * 2.0 ** -11 * top if fast else 0.0
        for out in (BF16, F32):
            z = mic.linear(x8, w8, x_scale=xs, w_scale=ws, out_dtype=out, fast_sums=fast)
            value, bound = R.linear(x8[rows], w8[cols], None, None, "none", out, xs[rows], ws[cols])[0]
            R.check(at(z, rows, cols), (value, bound + 1.01 * short(w8, ws)), "e4m3")
        _, gate, up = mic.gated_linear(x8, w8, u8, x_scale=xs, w_gate_scale=ws, w_up_scale=us, return_products=True,
                                       fast_sums=fast)
        ref = R.gated(x8[rows], w8[cols], u8[cols], "silu", BF16, xs[rows], ws[cols], us[cols])
        R.check(at(gate, rows, cols), (ref[1][0], ref[1][1] + 1.01 * short(w8, ws)), "e4m3 gate")
        R.check(at(up, rows, cols), (ref[2][0], ref[2][1] + 1.01 * short(u8, us)), "e4m3 up")


NORM = [(1, 1), (1, 4096), (3, 7), (5, 63), (2, 64), (7, 511), (4, 512), (9, 513), (3, 2048), (5, 2049), (2, 4096),
        (3, 4097), (2, 8192), (3, 8200), (2, 16384), (2, 20001), (700, 264), (300, 1000)]


@pytest.mark.parametrize("m,c", NORM)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rms_norm(m, c, dtype):
    x, res = values(1, m, c, dtype=dtype), values(2, m, c, std=2.0, dtype=dtype)
    w = values(3, c, std=0.1).add_(1).to(dtype)
    for residual in (None, res):
        for out in (dtype, E4M3):
            r = mic.rms_norm(x, w, residual=residual, eps=1e-6, out_dtype=out)
            want = R.rms_norm(x, w, residual, 1e-6, out)
            for key in want:
                R.check(getattr(r, key).float(), want[key], key)
            assert r.y.dtype is out and (r.scale is None) == (out is not E4M3)


@pytest.mark.parametrize("m,c", NORM)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rms_norm_backward(m, c, dtype):
    s, dy, dsum = (values(i, m, c, dtype=dtype) for i in (1, 2, 3))
    w = values(4, c, std=0.1).add_(1).to(dtype)
    rstd = (s.float().square().mean(1) + 1e-6).rsqrt()
    for extra in (None, dsum):
        dx, dw = mic.rms_norm_backward(dy, s, w, rstd, dsum=extra)
        ref = R.rms_norm_backward(dy, s, w, rstd, extra)
        R.check(dx, ref[0], "dx")
        R.check(dw, ref[1], "dweight")


def test_zero_lengths():
    for dtype in (F32, BF16):
        w, bias = values(1, 5, 0, dtype=dtype), values(2, 5, dtype=dtype)
        y = mic.linear(values(3, 4, 0, dtype=dtype), w, bias=bias, activation="relu")
        assert torch.equal(y, bias.clamp(min=0).expand(4, 5))                       # a sum of nothing
        assert mic.linear(values(3, 0, 8, dtype=dtype), values(4, 5, 8, dtype=dtype)).shape == (0, 5)
        assert mic.linear(values(3, 4, 8, dtype=dtype), values(4, 0, 8, dtype=dtype)).shape == (4, 0)
        h = mic.gated_linear(values(3, 4, 0, dtype=dtype), w, w)
        assert torch.equal(h, torch.zeros_like(h))
        dx, dw, db = mic.linear_backward(values(5, 0, 5, dtype=dtype), values(6, 0, 8, dtype=dtype),
                                         values(7, 5, 8, dtype=dtype), bias=True)
        assert dx.shape == (0, 8) and not dw.any() and dw.shape == (5, 8) and not db.any()
        dx, dg, du = mic.gated_linear_backward(*(values(i, *s, dtype=dtype) for i, s in enumerate(
            ((0, 5), (0, 8), (5, 8), (5, 8), (0, 5), (0, 5)))))
        assert dx.shape == (0, 8) and not dg.any() and not du.any()
        dx, dg, du = mic.gated_linear_backward(*(values(i, *s, dtype=dtype) for i, s in enumerate(
            ((6, 0), (6, 8), (0, 8), (0, 8), (6, 0), (6, 0)))))
        assert not dx.any() and dx.shape == (6, 8) and dg.shape == (0, 8)
        assert mic.rms_norm(values(1, 0, 8, dtype=dtype), values(2, 8, dtype=dtype)).y.shape == (0, 8)
        dx, dw = mic.rms_norm_backward(values(1, 0, 8, dtype=dtype), values(2, 0, 8, dtype=dtype),
                                       values(3, 8, dtype=dtype), values(4, 0))
        assert dx.shape == (0, 8) and not dw.any()


def test_norm_of_zero_rows_and_extremes():
    x = torch.zeros(3, 96, device=dev())
    x[1, 5] = 1e-30
    w = torch.ones(96, device=dev())
    r = mic.rms_norm(x, w, eps=1e-6, out_dtype=E4M3)
    assert not r.y[0].float().any() and r.scale[0] == 1 and not r.y[2].float().any()
    assert torch.isfinite(r.y.float()).all() and torch.isfinite(r.scale).all()
    assert r.y[1, 5].float() == 448.0
    x = values(1, 4, 96)
    x[2, 3] = float("nan")
    x[3, 4] = float("inf")
    r = mic.rms_norm(x, w)
    assert torch.isnan(r.y[2]).all() and torch.isfinite(r.y[:2]).all()          # a row keeps to itself
    assert torch.isnan(r.y[3, 4]) and not r.y[3, :4].any() and r.rstd[3] == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(3, 40, 72), (130, 96, 136), (300, 264, 200)])
def test_not_a_number_keeps_to_its_row(m, n, k, dtype):
    """What lies beside an operand, or in another row of it, never reaches a result."""
    x, w = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype)
    clean = mic.linear(x, w)
    xp, wp = pitched(x, 3, 1), pitched(w, 5, 3)                                   # NaN between and around the rows
    got = mic.linear(xp, wp)
    R.check(got, R.linear(x, w, None, None, "none", dtype)[0], "padded")
    x2 = x.clone()
    x2[m // 2] = float("inf")
    x2[m // 2, 0] = float("nan")
    y = mic.linear(x2, w)
    keep = torch.arange(m, device=dev()) != m // 2
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[m // 2]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 40, 72), (20, 96, 136), (150, 131, 77), (300, 264, 200)])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 1)])
def test_pitched_rows(m, n, k, pad, offset, dtype):
    def put(t):
        return pitched(t, pad, offset)
    x, w, wu = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype), values(3, n, k, dtype=dtype)
    dy, z, u = (values(i, m, n, dtype=dtype) for i in (4, 5, 6))
    R.check(mic.linear(put(x), put(w), residual=put(dy)), R.linear(x, w, None, dy, "none", dtype)[0], "y")
    R.check(mic.gated_linear(put(x), put(w), put(wu)), R.gated(x, w, wu, "silu", dtype)[0], "h")
    got = mic.linear_backward(put(dy), put(x), put(w), preact=put(z), activation="gelu", bias=True)
    for g, want in zip(got, R.linear_backward(dy, x, w, z, "gelu")):
        R.check(g, want, "linear backward")
    got = mic.linear_backward(put(dy), put(x), put(w))
    for g, want in zip(got[:2], R.linear_backward(dy, x, w, None, "none")):
        R.check(g, want, "linear backward, no activation")
    got = mic.gated_linear_backward(put(dy), put(x), put(w), put(wu), put(z), put(u))
    for g, want in zip(got, R.gated_backward(dy, x, w, wu, z, u, "silu")):
        R.check(g, want, "gated backward")
    weight = values(7, k, dtype=dtype)
    r = mic.rms_norm(put(x), weight, residual=put(x))
    for key, want in R.rms_norm(x, weight, x, 1e-6, dtype).items():
        R.check(getattr(r, key), want, key)
    got = mic.rms_norm_backward(put(x), put(r.sum), weight, r.rstd, dsum=put(x))
    for g, want in zip(got, R.rms_norm_backward(x, r.sum, weight, r.rstd, x)):
        R.check(g, want, "norm backward")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 33, 40), (70, 131, 65), (257, 264, 128)])
def test_writes_stay_inside_the_outputs(m, n, k, dtype):
    """Outputs with a pitch, through the C call: every cell between and around their rows keeps its value."""
    def out(rows, cols):
        base = torch.full((64 + rows * (cols + 5) + 64,), -7.0, dtype=dtype, device=dev())
        return base, base.as_strided((rows, cols), (cols + 5, 1), 64)

    def untouched(base, t):
        mask = torch.ones_like(base, dtype=torch.bool)
        mask.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(False)
        return bool((base[mask] == -7.0).all())

    code = {F32: 0, BF16: 2}[dtype]
    x, w, wu = values(1, m, k, dtype=dtype), values(2, n, k, dtype=dtype), values(3, n, k, dtype=dtype)
    dy, z, u = (values(i, m, n, dtype=dtype) for i in (4, 5, 6))
    h = mic.handle_for(x.device)
    mic.mic_set_stream(h, torch.cuda.current_stream().cuda_stream)

    def space(n_bytes):
        t = torch.full((n_bytes + 256,), 171, dtype=torch.uint8, device=dev())
        return t, t.data_ptr(), n_bytes

    (yb, y), (pb, p) = out(m, n), out(m, n)
    ws, wp, wn = space(mic.mic_linear_forward_workspace(h, code, m, n, k))
    mic.mic_linear_forward(h, code, code, mic.MIC_ACT_GELU, 0, m, n, k, x.data_ptr(), k, w.data_ptr(), k, 0, 0, 0, 0, 0,
                           y.data_ptr(), n + 5, p.data_ptr(), n + 5, wp, wn)
    ref = R.linear(x, w, None, None, "gelu", dtype)
    R.check(y, ref[0]), R.check(p, ref[1])
    assert untouched(yb, y) and untouched(pb, p) and bool((ws[wn:] == 171).all())

    (xb, dx), (gb, dg), (ub, du) = out(m, k), out(n, k), out(n, k)
    ws, wp, wn = space(mic.mic_gated_linear_backward_workspace(h, code, m, n, k))
    mic.mic_gated_linear_backward(h, code, mic.MIC_ACT_SILU, m, n, k, dy.data_ptr(), n, x.data_ptr(), k, w.data_ptr(), k,
                                  wu.data_ptr(), k, z.data_ptr(), n, u.data_ptr(), n, dx.data_ptr(), k + 5,
                                  dg.data_ptr(), k + 5, du.data_ptr(), k + 5, wp, wn)
    for got, want in zip((dx, dg, du), R.gated_backward(dy, x, w, wu, z, u, "silu")):
        R.check(got, want)
    assert untouched(xb, dx) and untouched(gb, dg) and untouched(ub, du) and bool((ws[wn:] == 171).all())

    (xb, dx), (gb, dg) = out(m, k), out(n, k)
    ws, wp, wn = space(mic.mic_linear_backward_workspace(h, code, m, n, k))
    db = torch.empty(n, dtype=dtype, device=dev())
    mic.mic_linear_backward(h, code, mic.MIC_ACT_RELU, m, n, k, dy.data_ptr(), n, x.data_ptr(), k, w.data_ptr(), k,
                            z.data_ptr(), n, dx.data_ptr(), k + 5, dg.data_ptr(), k + 5, db.data_ptr(), wp, wn)
    for got, want in zip((dx, dg, db), R.linear_backward(dy, x, w, z, "relu")):
        R.check(got, want)
    assert untouched(xb, dx) and untouched(gb, dg) and bool((ws[wn:] == 171).all())


def test_gradients_against_differences():
    """Central differences of the 64-bit forward forms, along random directions."""
    m, n, k, eps = 6, 20, 24, 1e-4
    x, w, wu, bias = values(1, m, k), values(2, n, k), values(3, n, k), values(4, n)
    dy = values(5, m, n)

    def along(f, t, grad, seed, what):
        v = values(seed, *t.shape).double().cpu()
        t64 = R.d(t)
        num = float(((f(t64 + eps * v) - f(t64 - eps * v)) * R.d(dy)).sum() / (2 * eps))
        got = float((R.d(grad) * v).sum())
        size = float((R.d(grad) * v).abs().sum())
        # the difference's own error: eps^2 times a third derivative of order 1 per term; the kernel's fp32 roundings
        assert abs(num - got) <= 1e-5 * size + 1e-6, (what, num, got)

    for name in ("gelu", "gelu_tanh", "silu"):
        y, z = mic.linear(x, w, bias=bias, activation=name, return_preact=True)
        dx, dw, db = mic.linear_backward(dy, x, w, preact=z, activation=name, bias=True)
        along(lambda t: R.act(t @ R.d(w).t() + R.d(bias), name), x, dx, 7, name)
        along(lambda t: R.act(R.d(x) @ t.t() + R.d(bias), name), w, dw, 8, name)
        along(lambda t: R.act(R.d(x) @ R.d(w).t() + t, name), bias, db, 9, name)
        h, gate, up = mic.gated_linear(x, w, wu, activation=name, return_products=True)
        dx, dg, du = mic.gated_linear_backward(dy, x, w, wu, gate, up, activation=name)
        along(lambda t: R.act(t @ R.d(w).t(), name) * (t @ R.d(wu).t()), x, dx, 10, name)
        along(lambda t: R.act(R.d(x) @ t.t(), name) * (R.d(x) @ R.d(wu).t()), w, dg, 11, name)
        along(lambda t: R.act(R.d(x) @ R.d(w).t(), name) * (R.d(x) @ t.t()), wu, du, 12, name)
    weight, dy = values(6, k), values(13, m, k)
    r = mic.rms_norm(x, weight)
    dx, dweight = mic.rms_norm_backward(dy, x, weight, r.rstd)

    def norm(s, g):
        return s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * g
    along(lambda t: norm(t, R.d(weight)), x, dx, 14, "norm")
    along(lambda t: norm(R.d(x), t), weight, dweight, 15, "norm weight")


def test_leading_dimensions_and_views():
    x = values(1, 3, 5, 64, dtype=BF16)
    w = values(2, 48, 64, dtype=BF16)
    y = mic.linear(x, w)
    assert y.shape == (3, 5, 48) and torch.equal(y.reshape(15, 48), mic.linear(x.reshape(15, 64), w))
    wide = values(3, 4, 6, 128, dtype=BF16)
    part = wide[..., 64:]                                      # one pitch of 128 over both leading dimensions
    assert torch.equal(mic.linear(part, w), mic.linear(part.contiguous(), w))
    r = mic.rms_norm(x, values(4, 64, dtype=BF16), out_dtype=E4M3)
    assert r.y.shape == x.shape and r.rstd.shape == (3, 5) and r.scale.shape == (3, 5)
    assert mic.linear(x[0, 0], w).shape == (48,)


def test_same_bits_again():
    for dtype in (F32, BF16):
        x, w, dy = values(1, 200, 1032, dtype=dtype), values(2, 300, 1032, dtype=dtype), values(3, 200, 300, dtype=dtype)
        first = mic.linear(x, w, activation="gelu")
        grads = mic.linear_backward(dy, x, w, preact=dy, activation="gelu", bias=True)
        for _ in range(3):
            assert torch.equal(first, mic.linear(x, w, activation="gelu"))
            assert all(torch.equal(a, b) for a, b in zip(grads, mic.linear_backward(dy, x, w, preact=dy,
                                                                                    activation="gelu", bias=True)))


def test_another_stream():
    x, w = values(1, 300, 520, dtype=BF16), values(2, 264, 520, dtype=BF16)
    want = mic.linear(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x2 = x * 2                                             # made on s: the call has to follow it there
        got = mic.linear(x2, w)
    s.synchronize()
    assert torch.equal(got, want * 2)                          # a power of two changes no rounding
    assert torch.equal(mic.linear(x, w), want)


def test_captured_block():
    """Norm, gated layer, linear layer and all their gradients in one graph, replayed on new inputs."""
    m, c, f = 96, 264, 520
    x, dy = values(1, m, c, dtype=BF16), values(2, m, c, dtype=BF16)
    weight = values(3, c, std=0.1).add_(1).to(BF16)
    wg, wu = values(4, f, c, std=0.06, dtype=BF16), values(5, f, c, std=0.06, dtype=BF16)
    wd = values(6, c, f, std=0.04, dtype=BF16)

    def step():
        r = mic.rms_norm(x, weight)
        h, gate, up = mic.gated_linear(r.y, wg, wu, return_products=True)
        y = mic.linear(h, wd, residual=x)
        dh, dwd, _ = mic.linear_backward(dy, h, wd)
        dn, dwg, dwu = mic.gated_linear_backward(dh, r.y, wg, wu, gate, up)
        dx, dweight = mic.rms_norm_backward(dn, r.sum, weight, r.rstd, dsum=dy)
        return y, dx, dweight, dwg, dwu, dwd

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(4):
        x.copy_(values(20 + i, m, c, dtype=BF16))
        dy.copy_(values(30 + i, m, c, dtype=BF16))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
