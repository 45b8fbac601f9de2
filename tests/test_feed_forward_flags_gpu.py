"""Arguments that say yes or no, where the native binding reads them."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic
from test_feed_forward_gpu import dev, values

pytestmark = pytest.mark.gpu


def test_a_tensor_is_no_flag():
    x, w, b, dy = values(1, 4, 8), values(2, 3, 8), values(3, 3), values(4, 4, 3)
    for call, name in ((lambda: mic.linear_backward(dy, x, w, bias=b), "bias"),
                       (lambda: mic.linear_backward(dy, x, w, bias=b[:1]), "bias"),
                       (lambda: mic.linear(x, w, return_preact=b), "return_preact"),
                       (lambda: mic.linear(x, w, fast_sums=b), "fast_sums"),
                       (lambda: mic.gated_linear(x, w, w, return_products=b), "return_products"),
                       (lambda: mic.gated_linear(x, w, w, fast_sums=b), "fast_sums")):
        with pytest.raises(TypeError, match=name):
            call()
    yes = torch.ones((), dtype=torch.bool, device=dev())                 # one bool is one wherever it lies
    assert torch.equal(mic.linear_backward(dy, x, w, bias=yes)[2], mic.linear_backward(dy, x, w, bias=1)[2])
    assert mic.linear_backward(dy, x, w, bias=0)[2] is None


def test_a_flag_without_a_truth_value_passes_its_error_on():
    class Neither:
        def __bool__(self):
            raise RuntimeError("neither")

    x, w, dy = values(1, 4, 8), values(2, 3, 8), values(4, 4, 3)
    for call in (lambda: mic.linear_backward(dy, x, w, bias=Neither()), lambda: mic.linear(x, w, fast_sums=Neither())):
        with pytest.raises(RuntimeError, match="neither"):
            call()
