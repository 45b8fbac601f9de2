"""GPU parity of e4m3 layers whose two scales multiply to what fp32 cannot hold, though the outputs fit.

Operands are whole numbers up to 3 times a power of two and scales have few bits, so every sum and every output is
exact in fp32: the only rounding is a bf16 output's own.
"""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
from test_feed_forward_gpu import BF16, E4M3, F32, dev, quantised, values

pytestmark = pytest.mark.gpu

# (x's scale, the weights', the operands' unit): scales whose product is past 2^128, below 2^-149 (it would be a zero),
# among the subnormals (it would lose its low bits), and a scale that is subnormal itself
PAIRS = [(2.0 ** 96, 2.0 ** 33, 2.0 ** -6), (2.0 ** -90, 2.0 ** -61, 128.0), (1.0625 * 2.0 ** -70, 1.03125 * 2.0 ** -76, 128.0),
         (1.625 * 2.0 ** -133, 2.0 ** 20, 16.0)]
# the vector units, the blocks, small tiles, split ones, whole and ragged large tiles
SIZES = [(1, 40, 64), (2, 33, 80), (20, 40, 96), (70, 65, 63), (40, 72, 2048), (512, 768, 128), (513, 1040, 264)]


def whole(seed, rows, cols, unit):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-3, 4, (rows, cols), generator=g).float() * unit


@pytest.mark.parametrize("xs,ws,unit", PAIRS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_scales_apart(m, n, k, xs, ws, unit):
    x, w, u = whole(1, m, k, unit), whole(2, n, k, unit), whole(3, n, k, unit)
    want, other = (x.double() @ t.double().t() * xs * ws for t in (w, u))
    x8, w8, u8 = (t.to(dev()).to(E4M3) for t in (x, w, u))
    sx, sw = (torch.full((size,), v, device=dev()) for size, v in ((m, xs), (n, ws)))
    for out in (F32, BF16):
        for fast in (False, True):
            y = mic.linear(x8, w8, x_scale=sx, w_scale=sw, out_dtype=out, fast_sums=fast)
            assert torch.equal(y.cpu(), want.to(out)), (out, fast)
    h, gate, up = mic.gated_linear(x8, w8, u8, activation="none", x_scale=sx, w_gate_scale=sw, w_up_scale=sw, out_dtype=F32,
                                   return_products=True)
    assert torch.equal(gate.cpu(), want.float()) and torch.equal(up.cpu(), other.float())
    assert torch.equal(h, gate * up)


@pytest.mark.parametrize("m,n,k", [(2, 40, 64), (20, 40, 96), (512, 768, 640), (513, 1040, 264)])
def test_few_scales_far_off(m, n, k):
    """One row and one column whose scales are far from the others', among tiles that have none such; bias and residual."""
    (x, xs), (w, ws) = quantised(1, m, k), quantised(2, n, k, std=k ** -0.5)
    xs[m // 2] = 2.0 ** -100
    ws[n // 3] = 2.0 ** 90
    for out in (F32, BF16):
        bias, res = values(3, n, dtype=out), values(4, m, n, dtype=out)
        y, z = mic.linear(x, w, bias=bias, residual=res, activation="relu", x_scale=xs, w_scale=ws, out_dtype=out,
                          return_preact=True)
        ref_y, ref_z = R.linear(x, w, bias, res, "relu", out, xs, ws)
        R.check(z, ref_z, "preact")
        R.check(y, ref_y, "y")
