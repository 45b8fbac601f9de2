"""What the feed-forward calls allocate and write beside their outputs."""
import re

import pytest
import torch

import convolution_forward_conv2d_amd as mic
import feed_forward_ref as R
from test_feed_forward_gpu import BF16, F32, dev, pitched, values

pytestmark = pytest.mark.gpu


def extra(call):
    """Bytes a call holds at most beside what it returns."""
    call()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = call()
    torch.cuda.synchronize()
    outputs = sum(t.numel() * t.element_size() for t in (out if isinstance(out, tuple) else (out,)) if t is not None)
    return torch.cuda.max_memory_allocated() - before - outputs


@pytest.mark.parametrize("pitch", [0, 8])
def test_aligned_rows_are_not_copied(pitch):
    m, n, k = 2048, 4096, 2304
    make = values if not pitch else lambda *a, **kw: pitched(values(*a, **kw), pitch)
    x, w, wu, dy, z = (make(i, *s, dtype=BF16) for i, s in enumerate(((m, k), (n, k), (n, k), (m, n), (m, n))))
    slack = 1 << 20                                            # the allocator's rounding
    dz, sums = m * n * 2, 1 << 23                              # and dbias's partial column sums

    def parts(name):
        """Partial sums of the products a name splits, on whole tiles: the larger of dx's and dw's."""
        most = 0
        for product, (rows, columns) in zip(name.split(", dw: "), ((m, k), (2 * n, k)) if "dw" in name else ((m, 2 * n),)):
            split = re.search(r"split (\d+)", product)
            most = max(most, int(split.group(1)) * rows * (columns + 255) // 256 * 256 * 4 if split else 0)
        return most

    assert extra(lambda: mic.linear(x, w, activation="gelu")) <= parts(mic.mic_linear_forward_kernel_name(None, 2, 2, 0, m, n, k)) + slack
    assert extra(lambda: mic.gated_linear(x, w, wu)) <= parts(mic.mic_gated_linear_forward_kernel_name(None, 2, 2, 0, m, n, k)) + slack
    plain, gelu = (parts(mic.mic_linear_backward_kernel_name(None, 2, a, m, n, k)) for a in (mic.MIC_ACT_NONE, mic.MIC_ACT_GELU))
    assert extra(lambda: mic.linear_backward(dy, x, w)) <= plain + sums + slack
    assert extra(lambda: mic.linear_backward(dy, x, w, preact=z, activation="gelu")) <= dz + gelu + sums + slack
    both = parts(mic.mic_gated_linear_backward_kernel_name(None, 2, m, n, k))
    assert extra(lambda: mic.gated_linear_backward(dy, x, w, wu, z, dy)) <= 2 * dz + both + slack


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(20, 264, 1024), (70, 128, 2048), (300, 520, 136), (513, 384, 264)])
def test_the_bytes_asked_for_are_enough(m, n, k, dtype):
    """Calls on aligned rows with exactly those bytes, the bytes behind them watched."""
    code = {F32: 0, BF16: 2}[dtype]
    x, w, wu = (values(i, *s, dtype=dtype) for i, s in enumerate(((m, k), (n, k), (n, k))))
    dy, z, u = (values(i, m, n, dtype=dtype) for i in (4, 5, 6))
    h = mic.handle_for(x.device)
    mic.mic_set_stream(h, torch.cuda.current_stream().cuda_stream)
    p = lambda t: t.data_ptr()

    def space(n_bytes):
        t = torch.full((n_bytes + 256,), 171, dtype=torch.uint8, device=dev())
        return t, p(t), n_bytes

    y, dx, dw, du, db = (torch.empty(s, dtype=dtype, device=dev()) for s in ((m, n), (m, k), (n, k), (n, k), (n,)))
    ws, wp, wn = space(mic.mic_linear_forward_workspace_aligned(h, code, m, n, k))
    mic.mic_linear_forward(h, code, code, 0, 0, m, n, k, p(x), k, p(w), k, 0, 0, 0, 0, 0, p(y), n, 0, 0, wp, wn)
    R.check(y, R.linear(x, w, None, None, "none", dtype)[0], "y")
    assert bool((ws[wn:] == 171).all())
    ws, wp, wn = space(mic.mic_gated_linear_forward_workspace_aligned(h, code, m, n, k))
    mic.mic_gated_linear_forward(h, code, code, mic.MIC_ACT_SILU, 0, m, n, k, p(x), k, p(w), k, p(wu), k, 0, 0, 0, p(y), n, 0, 0,
                                 0, 0, wp, wn)
    R.check(y, R.gated(x, w, wu, "silu", dtype)[0], "h")
    assert bool((ws[wn:] == 171).all())
    for act, name in ((mic.MIC_ACT_NONE, "none"), (mic.MIC_ACT_RELU, "relu")):
        ws, wp, wn = space(mic.mic_linear_backward_workspace_aligned(h, code, act, m, n, k))
        mic.mic_linear_backward(h, code, act, m, n, k, p(dy), n, p(x), k, p(w), k, p(z), n, p(dx), k, p(dw), k, p(db), wp, wn)
        for got, want in zip((dx, dw, db), R.linear_backward(dy, x, w, z, name)):
            R.check(got, want, name)
        assert bool((ws[wn:] == 171).all())
        if wn:
            with pytest.raises(mic.MicError) as e:
                mic.mic_linear_backward(h, code, act, m, n, k, p(dy), n, p(x), k, p(w), k, p(z), n, p(dx), k, p(dw), k, p(db), wp,
                                        wn - 1)
            assert e.value.status == mic.MIC_STATUS_BAD_PARAM
    ws, wp, wn = space(mic.mic_gated_linear_backward_workspace_aligned(h, code, m, n, k))
    mic.mic_gated_linear_backward(h, code, mic.MIC_ACT_SILU, m, n, k, p(dy), n, p(x), k, p(w), k, p(wu), k, p(z), n, p(u), n, p(dx),
                                  k, p(dw), k, p(du), k, wp, wn)
    for got, want in zip((dx, dw, du), R.gated_backward(dy, x, w, wu, z, u, "silu")):
        R.check(got, want, "gated")
    assert bool((ws[wn:] == 171).all())
