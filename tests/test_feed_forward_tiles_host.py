"""Which kernel a feed-forward product takes, without a GPU."""
import re

import pytest

import convolution_forward_conv2d_amd as mic
from feed_forward_tiles import BF16, E4M3, F32, cases, planned, product_of

CASES = list(cases())


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_a_case_runs_the_kernel_it_is_for(case):
    _, op, dtype, fast, m, n, k, aligned, name = case
    assert product_of(op, name, planned(op, dtype, fast, m, n, k, aligned)) == name
    if dtype == "e4m3":                                        # fp32 outputs take the same way
        assert planned(op, dtype, fast, m, n, k, aligned, out=F32) == name


def test_the_cases_reach_every_tile():
    large = ["256x256", "256x192", "192x256", "256x128", "128x256", "128x128"]
    small = ["128x128", "128x64", "64x128"]
    there = {(op, dtype, fast, re.sub(r" split \d+| pack.*", "", name)) for _, op, dtype, fast, _, _, _, _, name in CASES}
    for op in ("linear", "gated", "lb dx", "lb dw", "gb dx", "gb dw"):
        gradient = " " in op
        part = op.split()[1] + " " if gradient else ""
        for dtype, fast, tiles in (("bf16", False, large), ("f32", False, small), ("e4m3", True, large),
                                   ("e4m3", False, ["256x256", "256x192", "192x256", "128x128"])):
            if gradient and dtype == "e4m3":
                continue
            missing = [t for t in tiles if (op.split()[0], dtype, fast, part + "fast " + t) not in there]
            # two layers' weight gradients are one product of at least 128 rows, which 128 x 64 or 128 x 128 always suits
            assert missing == (["64x128"] if (op, dtype) == ("gb dw", "f32") else []), (op, dtype, missing)
            assert (op.split()[0], dtype, fast, part + "any 64x64") in there, (op, dtype)


def test_names():
    f = mic.mic_linear_forward_kernel_name
    assert f(None, BF16, BF16, 0, 8192, 4096, 9216) == "fast 256x256"
    assert f(None, BF16, BF16, 0, 1, 4096, 9216) == "few" and f(None, BF16, BF16, 0, 0, 8, 8) == "nothing"
    assert f(None, BF16, BF16, 0, 8192, 4096, 9216, False) == "fast 256x256 pack a pack b"
    # rows of 9218 bytes are not aligned wherever they start
    assert f(None, BF16, BF16, 0, 8192, 4096, 4609) == f(None, BF16, BF16, 0, 8192, 4096, 4609, False)
    g = mic.mic_linear_backward_kernel_name
    assert g(None, BF16, mic.MIC_ACT_GELU, 4096, 4096, 9216) == "dx: fast 256x192, dw: fast 256x192"
    assert g(None, BF16, mic.MIC_ACT_GELU, 0, 8, 8) .startswith("dx: nothing, dw: ")
    assert g(None, BF16, mic.MIC_ACT_GELU, 8, 0, 8).endswith("dw: nothing")
    assert mic.mic_gated_linear_backward_kernel_name(None, BF16, 4096, 9216, 4096) == "dx: fast 256x256, dw: fast 192x256"


def test_name_refusals():
    f, g = mic.mic_linear_forward_kernel_name, mic.mic_linear_backward_kernel_name
    for call, status in ((lambda: f(None, BF16, F32, 0, 4, 4, 4), mic.MIC_STATUS_NOT_SUPPORTED),
                         (lambda: f(None, BF16, BF16, 0, -4, 4, 4), mic.MIC_STATUS_BAD_PARAM),
                         (lambda: f(None, BF16, BF16, 0, 1 << 30, 4, 4), mic.MIC_STATUS_NOT_SUPPORTED),
                         (lambda: g(None, E4M3, 0, 4, 4, 4), mic.MIC_STATUS_NOT_SUPPORTED),
                         (lambda: g(None, BF16, 9, 4, 4, 4), mic.MIC_STATUS_NOT_SUPPORTED)):
        with pytest.raises(mic.MicError) as e:
            call()
        assert e.value.status == status
    import ctypes
    buf = ctypes.create_string_buffer(3)
    assert mic.lib().mic_linear_forward_kernel_name(None, BF16, BF16, 0, 8, 8, 8, 1, buf, 3) == mic.MIC_STATUS_BAD_PARAM
    assert mic.lib().mic_linear_forward_kernel_name(None, BF16, BF16, 0, 8, 8, 8, 1, None, 0) == mic.MIC_STATUS_BAD_PARAM
