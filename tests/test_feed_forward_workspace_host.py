"""Workspace sizes of the feed-forward operators, without a GPU."""
import ctypes
import random

import pytest

import convolution_forward_conv2d_amd as mic
from test_feed_forward_host import Handle

F32, BF16, E4M3 = mic.MIC_DTYPE_F32, mic.MIC_DTYPE_BF16, mic.MIC_DTYPE_F8_E4M3


@pytest.mark.parametrize("units", [32, 64, 128, 256])
def test_without_a_handle_a_workspace_is_enough_for_any(units):
    """The plan of a card's partition splits reductions elsewhere than the whole card's."""
    fields = Handle(0, units, None)
    h = ctypes.cast(ctypes.pointer(fields), ctypes.c_void_p)
    rng = random.Random(units)
    sizes = [(251, 4394, 4761)] + [tuple(int(2 ** rng.uniform(0, 13.2)) for _ in range(3)) for _ in range(300)]
    for m, n, k in sizes:
        for f, types in ((mic.mic_linear_forward_workspace, (F32, BF16, E4M3)), (mic.mic_gated_linear_forward_workspace, (BF16,)),
                         (mic.mic_linear_backward_workspace, (F32, BF16)), (mic.mic_gated_linear_backward_workspace, (BF16,))):
            for dtype in types:
                assert f(h, dtype, m, n, k) <= f(None, dtype, m, n, k), (f.__name__, dtype, m, n, k)
        assert mic.mic_rms_norm_backward_workspace(h, m, n) <= mic.mic_rms_norm_backward_workspace(None, m, n)


def pairs():
    """(bytes for aligned rows, for any) as functions of a handle, a type and m, n, k."""
    yield mic.mic_linear_forward_workspace_aligned, mic.mic_linear_forward_workspace, (F32, BF16, E4M3)
    yield mic.mic_gated_linear_forward_workspace_aligned, mic.mic_gated_linear_forward_workspace, (F32, BF16, E4M3)
    for act in (mic.MIC_ACT_NONE, mic.MIC_ACT_GELU):
        yield (lambda h, d, m, n, k, a=act: mic.mic_linear_backward_workspace_aligned(h, d, a, m, n, k),
               mic.mic_linear_backward_workspace, (F32, BF16))
    yield mic.mic_gated_linear_backward_workspace_aligned, mic.mic_gated_linear_backward_workspace, (F32, BF16)


def test_aligned_rows_are_not_copied():
    assert mic.mic_linear_forward_workspace_aligned(None, BF16, 8192, 4096, 9216) < 1 << 20
    assert mic.mic_gated_linear_forward_workspace_aligned(None, BF16, 8192, 4096, 9216) < 1 << 20
    # dz (a multiple of 64 columns a layer), and no copy of x, w or dz
    h = ctypes.cast(ctypes.pointer(Handle(0, 256, None)), ctypes.c_void_p)
    m, n, k = 4096, 9216, 4096
    dz = m * n * 2
    assert dz <= mic.mic_linear_backward_workspace_aligned(h, BF16, mic.MIC_ACT_GELU, m, n, k) < 1.3 * dz
    assert mic.mic_linear_backward_workspace_aligned(h, BF16, mic.MIC_ACT_NONE, m, n, k) < 0.3 * dz      # dz is dy
    assert 2 * dz <= mic.mic_gated_linear_backward_workspace_aligned(h, BF16, m, n, k) < 2.01 * dz
    # rows whose length is no multiple of 16 bytes are not aligned wherever they start
    assert (mic.mic_linear_forward_workspace_aligned(None, BF16, 4096, 4096, 4097)
            == mic.mic_linear_forward_workspace(None, BF16, 4096, 4096, 4097))


def test_aligned_rows_need_no_more():
    rng = random.Random(1)
    handles = [Handle(0, units, None) for units in (32, 64, 128, 256)]
    for _ in range(200):
        m, n, k = (int(2 ** rng.uniform(0, 13.2)) for _ in range(3))
        if rng.random() < 0.6:
            k = (k + 15) // 16 * 16
        for aligned, general, types in pairs():
            for d in types:
                most = aligned(None, d, m, n, k)
                assert most <= general(None, d, m, n, k), (d, m, n, k)
                for fields in handles:
                    h = ctypes.cast(ctypes.pointer(fields), ctypes.c_void_p)
                    assert aligned(h, d, m, n, k) <= most, (d, m, n, k, fields.num_cu)
                    assert aligned(h, d, m, n, k) <= general(h, d, m, n, k), (d, m, n, k, fields.num_cu)


def test_aligned_workspace_refusals():
    for call, status in ((lambda: mic.mic_linear_forward_workspace_aligned(None, BF16, -1, 4, 4), mic.MIC_STATUS_BAD_PARAM),
                         (lambda: mic.mic_linear_forward_workspace_aligned(None, mic.MIC_DTYPE_F64, 4, 4, 4), mic.MIC_STATUS_NOT_SUPPORTED),
                         (lambda: mic.mic_linear_backward_workspace_aligned(None, BF16, 7, 4, 4, 4), mic.MIC_STATUS_NOT_SUPPORTED),
                         (lambda: mic.mic_linear_backward_workspace_aligned(None, E4M3, 0, 4, 4, 4), mic.MIC_STATUS_NOT_SUPPORTED),
                         (lambda: mic.mic_gated_linear_backward_workspace_aligned(None, BF16, 4, 1 << 30, 4), mic.MIC_STATUS_NOT_SUPPORTED)):
        with pytest.raises(mic.MicError) as e:
            call()
        assert e.value.status == status
    assert mic.lib().mic_linear_forward_workspace_aligned(None, BF16, 4, 4, 4, None) == mic.MIC_STATUS_BAD_PARAM
