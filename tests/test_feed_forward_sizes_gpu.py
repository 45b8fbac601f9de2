"""GPU parity of the feed-forward operators on sizes past what one launch or one 32-bit count takes."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
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


@pytest.mark.parametrize("m", [1, 20, 300])
def test_offsets_past_32_bits(m, monkeypatch):
    """Weights of 2.4e9 elements: every way through a layer (few rows on the vector units and in blocks, large tiles) and
    its gradients, on sampled outputs, the first and last among them."""
    monkeypatch.setattr(R, "d", lambda t: None if t is None else t.detach().double())     # sums on the GPU
    n, k = (1 << 18) + 5, 9216
    g = torch.Generator(device=dev()).manual_seed(m)

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=BF16, device=dev()).normal_(std=std, generator=g)
    x, w = normal(m, k), normal(n, k, std=k ** -0.5)
    pick = torch.Generator().manual_seed(m)                    # 233016: 2^31 / k
    at = torch.cat([torch.tensor([0, 1, 233016, 233017, n - 2, n - 1]), torch.randint(0, n, (26,), generator=pick)]).to(dev())
    kat = torch.cat([torch.tensor([0, k - 1]), torch.randint(0, k, (30,), generator=pick)]).to(dev())
    y = mic.linear(x, w)
    R.check(y[:, at], R.linear(x, w[at], None, None, "none", BF16)[0], "y")
    h = mic.gated_linear(x, w, w)
    R.check(h[:, at], R.gated(x, w[at], w[at], "silu", BF16)[0], "h")
    del h
    dx, dw, db = mic.linear_backward(y, x, w, bias=True)
    ref = R.linear_backward(y[:, at], x[:, kat], w[at][:, kat], None, "none")
    R.check(dw[at][:, kat], ref[1], "dw")
    R.check(db[at], ref[2], "dbias")
    R.check(dx[:, kat], R.linear_backward(y, x[:, kat], w[:, kat], None, "none")[0], "dx")
