"""What a loss's gradient may be: a value, one per row, or a value that torch has expanded over the rows."""
import pytest
import torch

import convolution_forward_conv2d_amd as mic

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"


def values(seed, *shape, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lead", [(1,), (7,), (4, 6), (40, 1, 5)])
def test_expanded(lead, dtype):
    """The gradient of a sum of the rows' losses, as autograd makes it: the bits of the single value."""
    x, w, b = values(1, *lead, 40, dtype=dtype), values(2, 90, 40, std=0.3, dtype=dtype), values(3, 90, dtype=dtype)
    target = torch.randint(0, 90, lead, generator=torch.Generator().manual_seed(4)).to(DEV)
    got = mic.linear_cross_entropy(x, w, target, bias=b, reduction="none")
    loss = got.loss.requires_grad_()
    dloss, = torch.autograd.grad(0.75 * loss.sum(), loss)
    one = torch.tensor(0.75, device=DEV)
    assert dloss.shape == target.shape
    want = mic.linear_cross_entropy_backward(one, x, w, target, got.lse, bias=b)
    if target.numel() == 1:
        want = mic.linear_cross_entropy_backward(one.reshape(lead), x, w, target, got.lse, bias=b)
    for d in (dloss, one.expand(lead), torch.stack([one, one])[0].expand(lead)):
        for g, v in zip(mic.linear_cross_entropy_backward(d, x, w, target, got.lse, bias=b), want):
            assert torch.equal(g, v)


def test_refusals():
    x, w, t = values(1, 4, 6, 8), values(2, 5, 8), torch.zeros(4, 6, dtype=torch.int64, device=DEV)
    lse = mic.linear_cross_entropy(x, w, t).lse
    one = torch.ones((), device=DEV)
    for bad in (one.to(BF16).expand(4, 6), torch.ones(()).expand(4, 6), one.expand(24), one.expand(6, 4), torch.ones(6, device=DEV).expand(4, 6),
                torch.ones(4, 12, device=DEV)[:, ::2], torch.ones(4, 1, device=DEV).expand(4, 6)):
        with pytest.raises((ValueError, TypeError)):
            mic.linear_cross_entropy_backward(bad, x, w, t, lse)
