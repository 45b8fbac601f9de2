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
