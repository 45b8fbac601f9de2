"""Rows so many that a kernel's grid could pass what a launch takes, without a GPU."""
import re

import pytest

import convolution_forward_conv2d_amd as mic

F32, BF16, E4M3 = mic.MIC_DTYPE_F32, mic.MIC_DTYPE_BF16, mic.MIC_DTYPE_F8_E4M3
MOST = (1 << 30) - 1


def threads(name, m, columns):
    """The grid of a named kernel on m x columns outputs."""
    kernel, bm, bn = re.match(r"(fast|any) (\d+)x(\d+)", name).groups()
    split = re.search(r"split (\d+)", name)
    assert not split, "a split where tiles fill the card"
    return -(-m // int(bm)) * -(-columns // int(bn)) * (512 if kernel == "fast" else 256)


@pytest.mark.parametrize("m", [MOST, (1 << 29) + 1, 1 << 28, 1 << 24])
@pytest.mark.parametrize("n,k", [(1, 1), (1, 8), (1, 64), (64, 4), (65, 8), (128, 1), (128, 8)])
def test_a_product_takes_a_kernel_whose_grid_holds_it(m, n, k):
    for dtype, out in ((F32, F32), (BF16, BF16), (E4M3, BF16)):
        for aligned in (False, True):
            name = mic.mic_linear_forward_kernel_name(None, dtype, out, 0, m, n, k, aligned)
            assert threads(name, m, n) < 1 << 32, (dtype, aligned, name)
            if n <= 64:
                name = mic.mic_gated_linear_forward_kernel_name(None, dtype, out, 0, m, n, k, aligned)
                assert threads(name, m, (n + 15) // 16 * 32) < 1 << 32, (dtype, aligned, name)
    for dtype in (F32, BF16):
        dx = mic.mic_linear_backward_kernel_name(None, dtype, mic.MIC_ACT_RELU, m, k, n)[4:].split(", dw: ")[0]
        assert threads(dx, m, n) < 1 << 32, (dtype, dx)


def test_more_outputs_than_any_grid_holds_are_refused():
    """2^30 x 2^21 outputs are over four million GB; the call says so instead of failing at the launch."""
    with pytest.raises(mic.MicError) as e:
        mic.mic_linear_forward_kernel_name(None, BF16, BF16, 0, MOST, 1 << 21, 8)
    assert e.value.status == mic.MIC_STATUS_NOT_SUPPORTED
    assert mic.mic_linear_forward_workspace(None, BF16, MOST, 1 << 21, 8) == 0


def test_gated_sizes_are_refused_by_every_call_alike():
    """A gated layer's raw columns, twice its features, have to stay a 32-bit count: from 2^29 on no call takes them."""
    n = 1 << 29
    for call in (lambda: mic.mic_gated_linear_forward_workspace(None, BF16, 4, n, 4),
                 lambda: mic.mic_gated_linear_forward_workspace(None, BF16, 4, MOST, 4),
                 lambda: mic.mic_gated_linear_forward_workspace_aligned(None, BF16, 4, MOST, 8),
                 lambda: mic.mic_gated_linear_forward_kernel_name(None, BF16, BF16, 0, 4, MOST, 8),
                 lambda: mic.mic_gated_linear_backward_kernel_name(None, BF16, 4, MOST, 8),
                 lambda: mic.mic_linear_backward_kernel_name(None, BF16, 0, 4, n, 8)):
        with pytest.raises(mic.MicError) as e:
            call()
        assert e.value.status == mic.MIC_STATUS_NOT_SUPPORTED
