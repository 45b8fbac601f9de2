"""How much of a linear cross entropy's logits a workspace holds, from a few rows to millions: the limits the header states."""
import pytest

import convolution_forward_conv2d_amd as mic
from test_feed_forward_host import BF16, F32

LOGITS, GRADIENTS = 1 << 28, 1 << 29


def held(limit, m, classes, size):
    """Bytes of m rows of logits of `size` bytes: within the limit, or a thousand classes, or all of them."""
    return m * size * min((classes + 63) // 64 * 64, max(limit // (m * size), 1024))


# the unaligned features of the tall ones send their logits through memory
SIZES = [(1, 1, 1), (33, 130, 1001), (4096, 50021, 4096), (8192, 131072, 4096), (65536, 1030, 65), (65537, 1030, 65),
         (131073, 2049, 33), (224637, 628, 4325), (262145, 70000, 17), (295959, 447, 4883), (2068280, 770342, 3128)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype,size", [(F32, 4), (BF16, 2)])
@pytest.mark.parametrize("aligned", [False, True])
def test_limits(m, n, k, dtype, size, aligned):
    """A workspace is the logits or dz and, beside them, aligned copies of x and of the classes held, dx's fp32 sums, a row's
    statistics (12 bytes for 32 columns at least, for 8 of up to 32 rows) and column sums (4 bytes for 32 rows), and the parts
    of split products: at most 8 a CU of 256 x 256 fp32 (512 MB) or 256 parts of 4096 terms, never more than the output."""
    name = "_aligned" if aligned else ""
    forward = getattr(mic, "mic_linear_cross_entropy_workspace" + name)(None, dtype, m, n, k)
    backward = getattr(mic, "mic_linear_cross_entropy_backward_workspace" + name)(None, dtype, m, n, k)
    slack = (1 << 29) + 4096
    row = size * (k + 16)
    statistics = 12 * m * ((n + 7) // 8 if m <= 32 else (n + 31) // 32 + 1) + 8 * m
    assert forward <= held(LOGITS, m, n, 4) + row * (m + n) * 2 + statistics + slack
    classes = min(n, max(GRADIENTS // (m * size), 1024))
    dz = held(GRADIENTS, m, n, size)
    beside = row * (m + classes) * 2 + 4 * m * (k + 8) + 4 * (m // 32 + 1) * classes
    assert backward <= dz + dz * 4 // size + beside + slack


def test_tall_logits_pass_the_stated_bytes_by_a_thousand_classes():
    """So that each piece's reading of x serves a thousand classes, past 65536 rows a thousand of them are held, whatever
    they take: 538 MB of 224637 x 628."""
    name = mic.mic_linear_cross_entropy_kernel_name(None, BF16, 224637, 628, 4325, False)
    assert "fused" not in name and "1 pieces" in name
    held_bytes = mic.mic_linear_cross_entropy_workspace(None, BF16, 224637, 628, 4325)
    assert LOGITS < 224637 * 628 * 4 < held_bytes
