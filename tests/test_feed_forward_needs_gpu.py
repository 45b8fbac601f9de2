"""Gradients that are asked for alone: the bits of the call that computes them all, and None for the others."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
from test_feed_forward_gpu import BF16, F32, pitched, values

pytestmark = pytest.mark.gpu


def same(got, want, asked):
    for g, w, a in zip(got, want, asked):
        assert (g is None) == (not a)
        if a:
            assert torch.equal(g, w)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(5, 33, 40), (300, 264, 520), (0, 8, 16), (8, 0, 16)])
@pytest.mark.parametrize("pad", [0, 3])                        # through the native binding, and past it
def test_only_what_is_asked_for(m, n, k, dtype, pad):
    def put(t):
        return pitched(t, pad, 1) if pad and t.numel() else t
    x, w, wu = (put(values(i, *s, dtype=dtype)) for i, s in enumerate(((m, k), (n, k), (n, k))))
    dy, z, u = (put(values(i, m, n, dtype=dtype)) for i in (3, 4, 5))
    for act in ("none", "gelu"):
        want = mic.linear_backward(dy, x, w, preact=z, activation=act, bias=True)
        for dx in (False, True):
            for dw in (False, True):
                for bias in (False, True):
                    same(mic.linear_backward(dy, x, w, preact=z, activation=act, bias=bias, need_dx=dx, need_dw=dw), want,
                         (dx, dw, bias))
    want = mic.gated_linear_backward(dy, x, w, wu, z, u)
    for dx in (False, True):
        for dw in (False, True):
            same(mic.gated_linear_backward(dy, x, w, wu, z, u, need_dx=dx, need_dw=dw), want, (dx, dw, dw))
    s, g, weight = put(values(6, m, k, dtype=dtype)), put(values(7, m, k, dtype=dtype)), values(8, k, dtype=dtype)
    rstd = (s.float().square().mean(1) + 1e-6).rsqrt()
    want = mic.rms_norm_backward(g, s, weight, rstd)
    same(mic.rms_norm_backward(g, s, weight, rstd, need_dweight=False), want, (True, False))


def test_frozen_weights_cost_no_product():
    """dx alone allocates no gradient of the weights."""
    x, w, dy = values(1, 64, 2048, dtype=BF16), values(2, 4096, 2048, dtype=BF16), values(3, 64, 4096, dtype=BF16)
    mic.linear_backward(dy, x, w, need_dw=False)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    mic.linear_backward(dy, x, w, need_dw=False)
    torch.cuda.synchronize()
    asked = mic.mic_linear_backward_workspace_aligned(None, mic.MIC_DTYPE_BF16, mic.MIC_ACT_NONE, 64, 4096, 2048)
    assert torch.cuda.max_memory_allocated() - before <= x.numel() * 2 + asked + (1 << 20)


def test_flags_are_flags():
    x, w, dy = values(1, 4, 8), values(2, 3, 8), values(3, 4, 3)
    for call, name in ((lambda: mic.linear_backward(dy, x, w, need_dx=x), "need_dx"),
                       (lambda: mic.linear_backward(dy, x, w, need_dw=x), "need_dw"),
                       (lambda: mic.gated_linear_backward(dy, x, w, w, dy, dy, need_dw=x), "need_dw"),
                       (lambda: mic.rms_norm_backward(x, x, w[0], x[:, 0].contiguous(), need_dweight=x), "need_dweight")):
        with pytest.raises(TypeError, match=name):
            call()
