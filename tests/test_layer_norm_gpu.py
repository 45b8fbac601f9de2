"""GPU parity of layer norm and its gradient against plain 64-bit forms (bounds in training_ref)."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
import training_ref as T

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda:0"


def values(seed, *shape, std=1.0, mean=0.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).to(DEV)


def pitched(t, pad, offset=0):
    """t's values in rows `pad` elements further apart, `offset` elements into an allocation, NaN around them."""
    m, n = t.shape
    base = torch.full((offset + m * (n + pad) + 1,), float("nan"), dtype=F32, device=t.device).to(t.dtype)
    v = base.as_strided((m, n), (n + pad, 1), offset)
    v.copy_(t)
    return v


# one column, fewer than eight; each kernel's last width and the next: 512, 2048, 4096, 8192, 12288, 16384; rows cut at every place of
# a vector of eight
SIZES = [(1, 1), (1, 8), (3, 7), (5, 512), (2, 513), (4, 2048), (3, 2049), (2, 4096), (3, 4097), (2, 8192), (1, 8195),
         (2, 16384), (2, 16385), (1, 20001), (601, 300), (1030, 1001), (9, 510), (7, 1027), (4, 4092), (5, 8190), (3, 9213),
         (2, 12288), (2, 12295), (2, 14001)]


@pytest.mark.parametrize("m,c", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(m, c, dtype):
    x, w = values(1, m, c, dtype=dtype), values(2, c, std=0.2, mean=1.0, dtype=dtype)
    for bias, res, out in ((None, None, dtype), (values(3, c, dtype=dtype), values(4, m, c, std=2.0, mean=0.5, dtype=dtype), dtype),
                           (values(3, c, dtype=dtype), None, E4M3), (None, values(4, m, c, dtype=dtype), E4M3)):
        got = mic.layer_norm(x, w, bias=bias, residual=res, out_dtype=out)
        want = T.layer_norm(x, w, bias, res, 1e-5, out)
        assert got.y.dtype is out and got.y.shape == x.shape and got.mean.shape == got.rstd.shape == (m,)
        assert (got.scale is None) == (out is not E4M3)
        if res is None:
            assert got.sum is x
        for name in want:
            R.check(getattr(got, name), want[name], name)


@pytest.mark.parametrize("m,c", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward(m, c, dtype):
    s, w = values(1, m, c, std=1.5, mean=0.3, dtype=dtype), values(2, c, std=0.2, mean=1.0, dtype=dtype)
    dy = values(3, m, c, dtype=dtype)
    mean = s.float().mean(1)
    rstd = ((s.float() - mean[:, None]).square().mean(1) + 1e-5).rsqrt()
    for dsum, bias, weight in ((None, True, True), (values(4, m, c, dtype=dtype), False, True),
                               (None, True, False), (values(4, m, c, dtype=dtype), False, False)):
        dx, dw, db = mic.layer_norm_backward(dy, s, w, mean, rstd, dsum=dsum, bias=bias, need_dweight=weight)
        want = T.layer_norm_backward(dy, s, w, mean, rstd, dsum)
        R.check(dx, want[0], "dx")
        assert (dw is not None) == weight and (db is not None) == bias
        if weight:
            R.check(dw, want[1], "dweight")
        if bias:
            R.check(db, want[2], "dbias")


# more rows than one launch takes: workgroups walk them, each width its own kernel; the last few and next widths' ends cut
@pytest.mark.parametrize("m,c", [(769, 1), (801, 5), (2000, 8), (1100, 300), (800, 512), (900, 513), (800, 2048), (801, 2049),
                                 (800, 4096), (800, 4097), (769, 8192), (769, 8195), (800, 12288), (800, 12295), (769, 16384),
                                 (769, 16385), (769, 16400), (768, 4096), (768, 1001), (4097, 513), (5000, 1001), (4200, 1024),
                                 (4099, 520)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_of_many_rows(m, c, dtype):
    test_backward(m, c, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,c,pad,offset", [(3, 40, 8, 8), (5, 513, 3, 1), (7, 1001, 1, 3), (2, 16400, 5, 1)])
def test_pitches_and_alignments(m, c, pad, offset, dtype):
    x, res = (pitched(values(s, m, c, dtype=dtype), pad + s, offset) for s in (1, 2))
    w, b = values(3, c, dtype=dtype), values(4, c, dtype=dtype)
    got = mic.layer_norm(x, w, bias=b, residual=res)
    want = T.layer_norm(x, w, b, res, 1e-5, dtype)
    for name in want:
        R.check(getattr(got, name), want[name], name)
    got8 = mic.layer_norm(x, w, bias=b, residual=res, out_dtype=E4M3)
    want8 = T.layer_norm(x, w, b, res, 1e-5, E4M3)
    for name in want8:
        R.check(getattr(got8, name), want8[name], name)
    dy, dsum = (pitched(values(s, m, c, dtype=dtype), pad + s, offset) for s in (5, 6))
    dx, dw, db = mic.layer_norm_backward(dy, x, w, got.mean, got.rstd, dsum=dsum, bias=True)
    for g, v, name in zip((dx, dw, db), T.layer_norm_backward(dy, x, w, got.mean, got.rstd, dsum), ("dx", "dw", "db")):
        R.check(g, v, name)


@pytest.mark.parametrize("c", [300, 4096, 9000, 17000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_far_from_zero(c, dtype):
    """A variance from sums of squares would be lost here: values around 2000 with a spread of 0.5 (fp32) or 16 (bf16,
    whose steps are 8 there), one row with a single huge first value, one constant row."""
    x = values(1, 4, c, std=0.5 if dtype is F32 else 16.0, mean=2000.0, dtype=dtype)
    x[1, 0] = 30000.0
    x[2] = 7.0
    w, b = values(2, c, dtype=dtype), values(3, c, dtype=dtype)
    got = mic.layer_norm(x, w, bias=b)
    want = T.layer_norm(x, w, b, None, 1e-5, dtype)
    for name in want:
        R.check(getattr(got, name), want[name], name)
    assert torch.equal(got.y[2], b)                      # 7's sums and mean are exact: the distances are 0


def test_leading_dimensions_and_nothing():
    x = values(1, 2, 3, 5, 64, dtype=BF16)
    w = values(2, 64, dtype=BF16)
    got, flat = mic.layer_norm(x, w), mic.layer_norm(x.reshape(30, 64), w)
    assert got.y.shape == x.shape and got.mean.shape == (2, 3, 5) and torch.equal(got.y.reshape(30, 64), flat.y)
    none = mic.layer_norm(x[:0], w)
    assert none.y.shape == (0, 3, 5, 64)
    dx, dw, db = mic.layer_norm_backward(x[:0], x[:0], w, none.mean, none.rstd, bias=True)
    assert dx.shape == (0, 3, 5, 64) and not dw.any() and not db.any()


def test_no_number_stays_in_its_row():
    x, w = values(1, 5, 1000), values(2, 1000)
    clean = mic.layer_norm(x, w)
    x[1, 3], x[3, 999] = float("nan"), float("inf")
    got = mic.layer_norm(x, w)
    for r in (0, 2, 4):
        assert torch.equal(got.y[r], clean.y[r])
    assert got.y[1].isnan().all() and got.y[3].isnan().any() and got.mean[3].isinf()


def test_scale_of_zeros_and_small_rows():
    x = torch.zeros(2, 64, device=DEV)
    x[1] = values(1, 64) * 1e-20
    w = values(2, 64)
    got = mic.layer_norm(x, w, out_dtype=E4M3)
    assert float(got.scale[0]) == 1.0 and not got.y[0].float().any()
    want = T.layer_norm(x, w, None, None, 1e-5, E4M3)
    R.check(got.y[1:], tuple(v[1:] for v in want["y"]), "y")


def test_more_rows_than_a_launch_has_workgroups():
    """2^22 rows a launch: the next launch's rows, their sums and statistics at their places."""
    m = (1 << 22) + 5
    x = torch.zeros(m, 4, device=DEV)
    x[-7:] = values(1, 7, 4)
    res = torch.zeros_like(x)
    res[-7:] = values(2, 7, 4)
    w = values(3, 4)
    got = mic.layer_norm(x, w, residual=res, out_dtype=E4M3)
    want = T.layer_norm(x[-7:], w, None, res[-7:], 1e-5, E4M3)
    for name in want:
        R.check(getattr(got, name)[-7:], want[name], name)
    assert not got.sum[:-7].any()
    dx, dw, _ = mic.layer_norm_backward(got.sum, x, w, got.mean, got.rstd)
    assert dx.shape == x.shape and dw.isfinite().all()


def test_captured_and_replayed():
    """One capture holds forward and gradient; every replay has new inputs and the eager calls' bits."""
    x, res, w, b = values(1, 70, 1500, dtype=BF16), values(2, 70, 1500, dtype=BF16), values(3, 1500, dtype=BF16), values(4, 1500, dtype=BF16)

    def step():
        n = mic.layer_norm(x, w, bias=b, residual=res)
        return (n.y, n.sum, n.mean, n.rstd) + mic.layer_norm_backward(n.y, n.sum, w, n.mean, n.rstd, dsum=x, bias=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(values(10 + i, 70, 1500, dtype=BF16))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(out, want):
            assert torch.equal(a, e)


def test_another_stream_and_repeats():
    x, w = values(1, 333, 2000, dtype=BF16), values(2, 2000, dtype=BF16)
    first = mic.layer_norm(x, w)
    grads = mic.layer_norm_backward(x, x, w, first.mean, first.rstd, bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = mic.layer_norm(x, w)
        again = mic.layer_norm_backward(x, x, w, other.mean, other.rstd, bias=True)
    s.synchronize()
    assert torch.equal(first.y, other.y)
    for a, b in zip(grads, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [4104, 4101])
def test_offsets_past_32_bits(cols):
    """More than 2^32 elements: the last rows' results, bit for bit, are those of a call on them alone
    (on more rows than one launch takes, as all are)."""
    rows = (1 << 20) + 5
    x = torch.empty(rows, cols, dtype=BF16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    w, b = values(2, cols, dtype=BF16), values(3, cols, dtype=BF16)
    r = mic.layer_norm(x, w, bias=b)
    last = mic.layer_norm(x[-1000:], w, bias=b)
    for name in ("y", "mean", "rstd"):
        assert torch.equal(getattr(r, name)[-1000:], getattr(last, name)), name
    dx = mic.layer_norm_backward(x, r.sum, w, r.mean, r.rstd, need_dweight=False)[0]
    assert torch.equal(dx[-1000:], mic.layer_norm_backward(x[-1000:], last.sum, w, last.mean, last.rstd, need_dweight=False)[0])


def test_refusals():
    x, w = values(1, 4, 8), values(2, 8)
    mean = x.mean(1)
    for bad in (dict(weight=w[:7]), dict(weight=w.double()), dict(bias=w[:7]), dict(bias=w.to(BF16)), dict(residual=x[:3]),
                dict(residual=x.to(BF16)), dict(eps=-1.0), dict(eps=float("nan")), dict(out_dtype=BF16), dict(x=x.t()),
                dict(x=x.cpu()), dict(weight=w.cpu()), dict(x=x.long()), dict(x=x[:, :0], weight=w[:0])):
        with pytest.raises((ValueError, TypeError)):
            mic.layer_norm(**dict(dict(x=x, weight=w), **bad))
    for bad in (dict(sum=x[:3]), dict(mean=mean[:3]), dict(rstd=mean.to(BF16)), dict(dsum=x.to(BF16)), dict(bias=x),
                dict(need_dweight=x), dict(weight=w[:4])):
        with pytest.raises((ValueError, TypeError)):
            mic.layer_norm_backward(**dict(dict(dy=x, sum=x, weight=w, mean=mean, rstd=mean), **bad))
