"""What the linear cross entropy rounds: the gradient of the logits of bf16 tensors, and the exponentials of its rows' sums."""
import math

import pytest
import torch

import convolution_forward_conv2d_amd as mic
import training_ref as T

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DEV = "cuda:0"
U = 2.0 ** -24


def values(seed, *shape, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


# dz in the tiles that make the logits, of logits in memory
@pytest.mark.parametrize("m,n,k", [(1024, 4000, 256), (128, 130, 1024)])
@pytest.mark.parametrize("low,high", [(0.1, 0.1), (0.5, 0.5), (0.9, 0.9), (0.1, 0.9)])
@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_targets_with_a_probability(m, n, k, low, high, each, dtype):
    """A network past its first steps: rows whose target has probability `low` to `high`, so that its share of dz, p - 1,
    takes a rounding of its own, half a step of bf16 (counted in the bounds), with one dloss and one per row."""
    x, w = values(1, m, k, dtype=dtype), values(2, n, k, std=2 * k ** -0.5, dtype=dtype)
    target = torch.randint(0, n, (m,), generator=torch.Generator().manual_seed(3)).to(DEV)
    want = torch.logit(torch.linspace(low, high, m, dtype=torch.float64, device=DEV))
    along = w[target].double()
    along /= along.square().sum(1, keepdim=True)
    for _ in range(6):
        p = torch.softmax(x.double() @ w.double().t(), 1).gather(1, target[:, None])[:, 0]
        x = (x.double() + (want - torch.logit(p.clamp(1e-15, 1 - 1e-12)))[:, None] * along).to(dtype)
    got = mic.linear_cross_entropy(x, w, target, reduction="none" if each else "mean")
    dloss = values(4, m).abs() + 0.5 if each else torch.tensor(1.2375, device=DEV)
    grads = mic.linear_cross_entropy_backward(dloss, x, w, target, got.lse, count=got.count)
    ref = T.cross_entropy_backward(dloss, x, w, None, target, got.lse, got.count)
    for g, r, name in zip(grads, ref, ("dx", "dw")):
        T.check(g, r, name)


# rows of 8 columns a run (few rows), 32 to 96 (tiles), and in memory
@pytest.mark.parametrize("m,n", [(1, 65536), (20, 4000), (260, 135), (515, 20011), (1000, 8200), (128, 1000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_exponentials(m, n, dtype):
    """Logits that are exact, of which most of a sum is as far from its run's largest as a sum can be.

    A sum's exponentials are off by 2 U (the hardware's) and, of bf16 tensors, 1.23 U of their argument's size (its
    rounding, and log2 e's), which in a sum over n terms weighs d - 1 at most, d - 1 = (n - 1) e^-d: 2.6 at 96 columns,
    3.2 U in all; fp32 ones by 4 U (2^-22).  Two exponentials of 4 U join lanes and runs; 96 + n / 1000 additions one
    after the other; the logarithm 2 U of itself and 1 U of the sum's error, lse a rounding of itself."""
    k = 8
    far = torch.arange(n) % 96 != 5                            # one near class in every 96
    w = torch.zeros(n, k, dtype=dtype)
    w[:, 0], w[:, 1] = torch.where(far, -3.609375, 0.0), 0.0078125 * (torch.arange(n) % 3)
    x = torch.zeros(m, k, dtype=dtype)
    x[:, :2] = 1
    target = torch.zeros(m, dtype=torch.int64)
    got = mic.linear_cross_entropy(x.to(DEV), w.to(DEV), target.to(DEV), reduction="none")
    z = (x[:1].double() @ w.double().t())[0]
    lse = float(torch.logsumexp(z, 0))
    off = (2 + 4 + 2 * 4 + 96 + n / 1000 + 2 * math.log(n) + 2 * abs(lse)) * U
    assert float((got.lse.double() - lse).abs().max()) <= off
    loss = lse - float(z[0])
    assert float((got.loss.double() - loss).abs().max()) <= off + 4 * U * (abs(loss) + 4)
