"""What the operators allocate is torch's to see: by dispatch modes and profilers, and to fill under deterministic algorithms."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import convolution_forward_conv2d_amd as mic

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
DEV = "cuda:0"


def calls():
    """(name, call, tensors it allocates for its results) of every operator whose contiguous arguments go through the binding."""
    g = torch.Generator().manual_seed(1)
    x, w, u = (torch.randn(s, generator=g).to(BF16).to(DEV) for s in ((8, 64), (48, 64), (48, 64)))
    h, d = torch.randn(8, 48, generator=g).to(BF16).to(DEV), torch.ones((), device=DEV)
    v = torch.ones(64, dtype=BF16, device=DEV)
    t = torch.zeros(8, dtype=torch.int64, device=DEV)
    n, r = mic.layer_norm(x, v), mic.rms_norm(x, v)
    y, gate, up = mic.gated_linear(x, w, u, return_products=True)
    loss = mic.linear_cross_entropy(x, w, t)
    return [("rms_norm", lambda: mic.rms_norm(x, v, residual=x), 3), ("rms_norm_backward", lambda: mic.rms_norm_backward(x, x, v, r.rstd), 2),
            ("linear", lambda: mic.linear(x, w), 1), ("linear_backward", lambda: mic.linear_backward(h, x, w), 2),
            ("gated_linear", lambda: mic.gated_linear(x, w, u), 1),
            ("gated_linear_backward", lambda: mic.gated_linear_backward(h, x, w, u, gate, up), 3),
            ("layer_norm", lambda: mic.layer_norm(x, v, residual=x), 4),
            ("layer_norm_backward", lambda: mic.layer_norm_backward(x, x, v, n.mean, n.rstd), 2),
            ("dropout", lambda: mic.dropout(x, 0.5, 1), 1),
            ("linear_cross_entropy", lambda: mic.linear_cross_entropy(x, w, t), 3),
            ("linear_cross_entropy_backward", lambda: mic.linear_cross_entropy_backward(d, x, w, t, loss.lse, count=loss.count), 2)]


class Names(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.seen.append(str(func))
        return func(*args, **(kwargs or {}))


def tensors(result):
    return [t for t in (result if isinstance(result, (tuple, list)) else (result,)) if t is not None]


def test_dispatch_modes():
    for name, call, count in calls():
        plain = tensors(call())
        with Names() as names:
            got = tensors(call())
        assert sum("aten.empty" in n for n in names.seen) >= count, (name, names.seen)
        for a, b in zip(got, plain):
            assert torch.equal(a, b) and a.shape == b.shape and a.dtype is b.dtype and a.device == b.device, name


def test_deterministic_algorithms():
    """Uninitialised memory is filled, and the results are the same."""
    for name, call, count in calls():
        plain = tensors(call())
        torch.use_deterministic_algorithms(True)
        try:
            with torch.autograd.profiler.profile(use_device=None) as p:
                got = tensors(call())
        finally:
            torch.use_deterministic_algorithms(False)
        fills = sum(e.name == "aten::fill_" for e in p.function_events)
        assert fills >= count, (name, fills)
        for a, b in zip(got, plain):
            assert torch.equal(a, b), name
