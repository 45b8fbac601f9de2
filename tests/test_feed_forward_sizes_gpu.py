"""GPU parity of the feed-forward operators on sizes past what one launch or one 32-bit count takes."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
from test_feed_forward_gpu import BF16, E4M3, F32, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,c", [((1 << 26) + 5, 8), ((1 << 24) + 3, 520)])
def test_norm_of_more_rows_than_a_grid_takes(m, c):
    """A workgroup per row: 2^26 of 64 threads, or 2^24 of 256, are 2^32 threads.  A row does not depend on its
    neighbours, so every result is that of a short call on the same rows, bit for bit."""
    g = torch.Generator(device=dev()).manual_seed(1)
    x = torch.empty((m, c), dtype=BF16, device=dev()).normal_(generator=g)
    weight = torch.empty(c, dtype=BF16, device=dev()).normal_(generator=g)
    starts = [0, (1 << 22) - 3, (1 << 23) - 3, (1 << 24) - 6, (1 << 25) - 3, (1 << 26) - 4, m - 7]
    for out, residual in ((BF16, None), (E4M3, x)):
        r = mic.rms_norm(x, weight, residual=residual, out_dtype=out)
        for a in starts:
            if a + 7 > m:
                continue
            rows = slice(a, a + 7)
            want = mic.rms_norm(x[rows], weight, residual=None if residual is None else x[rows], out_dtype=out)
            assert torch.equal(r.rstd[rows], want.rstd), a
            assert torch.equal(r.y[rows].float(), want.y.float()), a
            assert torch.equal(r.sum[rows], want.sum), a
            if out is E4M3:
                assert torch.equal(r.scale[rows], want.scale), a
        del r


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_as_many_rows_as_there_may_be(dtype):
    """2^30 - 1 rows of one feature: 2^24 tiles of 64 rows would be 2^32 threads.  An output is one product, rounded once."""
    m = (1 << 30) - 1
    x = torch.empty((m, 1), dtype=dtype, device=dev()).normal_(generator=torch.Generator(device=dev()).manual_seed(2))
    w = torch.tensor([[1.25]], dtype=dtype, device=dev())
    y = mic.linear(x, w)
    for a in range(0, m, 1 << 27):
        rows = slice(a, min(a + (1 << 27), m))
        assert torch.equal(y[rows], (x[rows].float() * 1.25).to(dtype)), a
