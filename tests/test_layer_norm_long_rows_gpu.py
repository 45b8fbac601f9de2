"""Layer norm on rows too long for the registers, more of them than one launch takes (or, of the gradient, has workgroups)."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
import training_ref as T

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda:0"
LAUNCH = 1 << 16


def values(seed, *shape, dtype=F32):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=g)


@pytest.mark.parametrize("c", [12296, 12291])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (BF16, E4M3)])
def test_next_launch(c, dtype, out):
    """Around the seam and at both ends every result holds against 64 bits; all rows have the bits of smaller calls."""
    m = LAUNCH + 9
    x, res, w, b = values(1, m, c, dtype=dtype), values(2, m, c, dtype=dtype), values(3, c, dtype=dtype), values(4, c, dtype=dtype)
    got = mic.layer_norm(x, w, bias=b, residual=res, out_dtype=out)
    rows = [0, 1, LAUNCH - 2, LAUNCH - 1, LAUNCH, LAUNCH + 1, m - 1]
    want = T.layer_norm(x[rows], w, b, res[rows], 1e-5, out)
    for name in want:
        R.check(getattr(got, name)[rows], want[name], name)
    for part in (slice(0, 1000), slice(LAUNCH - 1000, m)):
        alone = mic.layer_norm(x[part], w, bias=b, residual=res[part], out_dtype=out)
        for name in want:
            assert torch.equal(getattr(got, name)[part].float(), getattr(alone, name).float()), name


def test_next_launch_of_apart_rows_alone():
    """A pitch, no residual, no bias: no sum is written."""
    m, c = LAUNCH + 3, 12290
    x = torch.full((m, c + 6), float("nan"), dtype=BF16, device=DEV)[:, :c]
    x.normal_(generator=torch.Generator(DEV).manual_seed(1))
    w = values(2, c, dtype=BF16)
    got = mic.layer_norm(x, w)
    assert got.sum is x
    rows = [0, LAUNCH - 1, LAUNCH, m - 1]
    want = T.layer_norm(x[rows], w, None, None, 1e-5, BF16)
    for name in ("y", "mean", "rstd"):
        R.check(getattr(got, name)[rows], want[name], name)


@pytest.mark.parametrize("c", [16392, 16387])
def test_gradient_walks(c):
    """Workgroups of the gradient's one launch that have a second row."""
    m, few = LAUNCH + 7, 40
    s, dsum, w = values(1, m, c, dtype=BF16), values(2, m, c, dtype=BF16), values(3, c, dtype=BF16)
    dy = torch.zeros(m, c, dtype=BF16, device=DEV)             # gradients in the first and last rows alone
    ends = torch.cat([torch.arange(few), torch.arange(m - few, m)]).to(DEV)
    dy[ends] = values(4, 2 * few, c, dtype=BF16)
    mean, rstd = values(5, m) * 0.1, values(6, m).abs() + 0.5
    dx, dw, db = mic.layer_norm_backward(dy, s, w, mean, rstd, dsum=dsum, bias=True)
    want = T.layer_norm_backward(dy[ends], s[ends], w, mean[ends], rstd[ends], dsum[ends])
    for got, v, name in ((dx[ends], want[0], "dx"), (dw, want[1], "dweight"), (db, want[2], "dbias")):
        R.check(got, v, name)
    rest = slice(few, m - few)
    for first in range(few, m - few, 8192):
        part = slice(first, min(first + 8192, rest.stop))
        assert torch.equal(dx[part], dsum[part])               # without dy what reaches sum past the norm
