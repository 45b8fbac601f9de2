"""GPU parity of dropout against the generator in 64-bit integers on the host."""
import numpy as np
import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
import training_ref as T

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"
SEED, OFFSET = 0x0123456789abcdef, 0xfedcba9876543210


def values(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5), (2, 3, 513), (128, 4096), (511, 1001), (4, 3, 13, 13)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p", [0.1, 0.5, 0.875])
def test_contiguous(shape, dtype, p):
    x, res = values(1, *shape, dtype=dtype), values(2, *shape, dtype=dtype)
    for r in (None, res):
        y = mic.dropout(x, p, SEED, offset=OFFSET, residual=r)
        want, kept = T.dropout(x, p, SEED, OFFSET, r)
        assert y.dtype is dtype and y.shape == x.shape
        R.check(y, want, "y")
        assert torch.equal(y.cpu()[~kept], (torch.zeros_like(x) if r is None else r).cpu()[~kept])
    assert torch.equal(mic.dropout_backward(res, p, SEED, offset=OFFSET), mic.dropout(res, p, SEED, offset=OFFSET))


@pytest.mark.parametrize("m,c,pad,start", [(5, 8, 8, 0), (4, 7, 1, 1), (9, 3, 2, 1), (33, 1001, 7, 5), (70, 512, 64, 0), (3, 1, 4, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_apart(m, c, pad, start, dtype):
    """The mask goes by the position in the tensor, not in memory; what lies between rows stays."""
    def apart(t):
        v = torch.full((start + m * (c + pad) + 3,), float("nan"), dtype=dtype, device=DEV).as_strided((m, c), (c + pad, 1), start)
        return v.copy_(t)

    x, res = values(1, m, c, dtype=dtype), values(2, m, c, dtype=dtype)
    want = mic.dropout(x, 0.3, 5, residual=res)
    assert torch.equal(mic.dropout(apart(x), 0.3, 5, residual=apart(res)), want)
    assert torch.equal(mic.dropout(x, 0.3, 5, residual=apart(res)), want)
    assert torch.equal(mic.dropout(apart(x), 0.3, 5, residual=res), want)
    # into rows apart, and in place, by the C call
    out = torch.full((m, c + pad), -5.0, dtype=dtype, device=DEV)
    h = mic.handle_for()
    mic.mic_set_stream(h, torch.cuda.current_stream().cuda_stream)
    code = {F32: mic.MIC_DTYPE_F32, BF16: mic.MIC_DTYPE_BF16}[dtype]
    mic.mic_dropout(h, code, m, c, 0.3, 5, 0, None, x.data_ptr(), c, res.data_ptr(), c, out.data_ptr(), c + pad)
    assert torch.equal(out[:, :c], want) and bool((out[:, c:] == -5.0).all())
    inside = x.clone()
    mic.mic_dropout(h, code, m, c, 0.3, 5, 0, None, inside.data_ptr(), c, res.data_ptr(), c, inside.data_ptr(), c)
    assert torch.equal(inside, want)


def test_edges_of_p():
    x = values(1, 1000)
    assert torch.equal(mic.dropout(x, 0.0, 1), x)
    assert torch.equal(mic.dropout(x, 2.0 ** -18, 1), x)         # below half of 2^-16: none
    assert not mic.dropout(x, 1.0, 1).any() and not mic.dropout(x, 1, 1).any()
    assert torch.equal(mic.dropout(x, 1.0, 1, residual=x), x)
    # the scale is that of p as it is rounded
    y = mic.dropout(torch.ones(4096, device=DEV), 0.3, 9)
    assert float(y.max()) == np.float32(65536 / (65536 - round(0.3 * 65536)))


def test_dropped_values_leave_no_trace():
    x = values(1, 4096)
    _, kept = T.dropout(x, 0.5, 3, 0, None)
    x[~kept.to(DEV)] = float("nan")
    y = mic.dropout(x, 0.5, 3)
    assert y.isfinite().all() and not y.cpu()[~kept].any()
    x[~kept.to(DEV)] = float("-inf")
    assert torch.equal(mic.dropout(x, 0.5, 3), y)


def test_share_and_independence():
    """Of 2^20 lots a share p is dropped, within five standard deviations; seeds, offsets and neighbours share no mask."""
    n, p = 1 << 20, 0.1
    x = torch.ones(n, device=DEV)
    masks = [mic.dropout(x, p, s, offset=o) == 0 for s, o in ((1, 0), (2, 0), (1, 1), (1 << 32, 0), (1, 1 << 32))]
    masks.append(masks[0].roll(1))
    q, tol = round(p * 65536) / 65536, 5 * (0.09 / n) ** 0.5
    for i, a in enumerate(masks):
        assert abs(float(a.float().mean()) - q) < tol
        for b in masks[i + 1:]:
            assert abs(float((a & b).float().mean()) - q * q) < 5 * (q * q / n) ** 0.5


def test_seed_in_device_memory():
    x = values(1, 300, 40)
    assert torch.equal(mic.dropout(x, np.float32(0.5), np.int64(7), offset=np.int32(3)), mic.dropout(x, 0.5, 7, offset=3))
    state = torch.tensor([77, 1000], device=DEV)
    assert torch.equal(mic.dropout(x, 0.4, state, offset=5), mic.dropout(x, 0.4, 77, offset=1005))
    assert torch.equal(mic.dropout_backward(x, 0.4, state, offset=5), mic.dropout_backward(x, 0.4, 77, offset=1005))
    state.copy_(torch.tensor([-2, -1], device=DEV))              # as 64-bit patterns
    assert torch.equal(mic.dropout(x, 0.4, state, offset=3), mic.dropout(x, 0.4, (1 << 64) - 2, offset=2))


def test_captured_draws_anew():
    x = values(1, 50, 999, dtype=BF16)
    state = torch.tensor([7, 0], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mic.dropout(x, 0.2, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mic.dropout(x, 0.2, state, offset=2, residual=x)
        dx = mic.dropout_backward(y, 0.2, state, offset=2)
    for i in range(4):
        state.copy_(torch.tensor([7, 10 * i], device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = mic.dropout(x, 0.2, 7, offset=10 * i + 2, residual=x)
        assert torch.equal(y, want) and torch.equal(dx, mic.dropout_backward(want, 0.2, 7, offset=10 * i + 2))


def test_positions_past_32_bits():
    """A tensor of more than 2^32 elements: the last ones' lots are those of their own positions."""
    n = (1 << 32) + 40
    x = torch.ones(n, dtype=BF16, device=DEV)
    y = mic.dropout(x, 0.5, 11)
    first = (1 << 32) - 64
    want = torch.from_numpy(T.lots(104, 11, 0, first=first) >= 32768)
    assert torch.equal(y[first:].cpu() != 0, want)
    assert not torch.equal(y[:40], y[1 << 32:])


def test_nothing():
    assert mic.dropout(torch.zeros(0, 5, device=DEV), 0.1, 1).shape == (0, 5)


def test_refusals():
    x = values(1, 4, 8)
    for bad in (dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(seed=-1), dict(seed=1 << 64), dict(seed=1.5), dict(seed=True),
                dict(seed=torch.zeros(2, device=DEV)), dict(seed=torch.zeros(2, dtype=torch.int64)),
                dict(seed=torch.zeros(3, dtype=torch.int64, device=DEV)), dict(offset=-1), dict(offset=1 << 64),
                dict(residual=x[:3]), dict(residual=x.to(BF16)), dict(residual=x.cpu()), dict(x=x.double()), dict(x=x.cpu()),
                dict(x=x.t()), dict(x=x[:, ::2]), dict(p=x)):
        with pytest.raises((ValueError, TypeError)):
            mic.dropout(**dict(dict(x=x, p=0.5, seed=1), **bad))
