"""Arguments that say yes or no, without a GPU."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic


def test_a_tensor_is_no_flag():
    x, w, b = torch.zeros(4, 8), torch.zeros(3, 8), torch.zeros(3)
    dy = torch.zeros(4, 3)
    for call, name in ((lambda: mic.linear_backward(dy, x, w, bias=b), "bias"),
                       (lambda: mic.linear_backward(dy, x, w, bias=b[:1]), "bias"),
                       (lambda: mic.linear(x, w, return_preact=b), "return_preact"),
                       (lambda: mic.linear(x, w, fast_sums=b), "fast_sums"),
                       (lambda: mic.gated_linear(x, w, w, return_products=b), "return_products"),
                       (lambda: mic.gated_linear(x, w, w, fast_sums=b), "fast_sums")):
        with pytest.raises(TypeError, match=name):
            call()
