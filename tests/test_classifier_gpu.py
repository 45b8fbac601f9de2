"""Layer norm, the gated and linear layers, dropout and the cross entropy run together, eager and captured, as a classifier
trains: its gradients against 64-bit ones."""
import os
import sys

import pytest
import torch

import convolution_forward_conv2d_amd as mic
import training_ref as T

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import classifier as C  # noqa: E402

DEV = "cuda:0"
ROWS, WIDTH, HIDDEN, CLASSES = 70, 96, 136, 203


def gradients64(model, x, target, seed, offset):
    """(loss, gradients of the weights, gradient of x) by autograd in float64 on the host, with the same masks."""
    w = {k: v.detach().cpu().double().requires_grad_() for k, v in model.w.items()}
    x = x.detach().cpu().double().requires_grad_()

    def norm(v, weight, bias):
        apart = v - v.mean(1, keepdim=True)
        return apart / torch.sqrt(apart.square().mean(1, keepdim=True) + 1e-5) * weight + bias

    least = round(model.drop * 65536)
    kept = torch.from_numpy(T.lots(x.numel(), seed, offset) >= least).reshape(x.shape).double() * (65536 / (65536 - least))
    n = norm(x, w["norm"], w["norm_bias"])
    gate = n @ w["gate"].t()
    s = x + (gate * torch.sigmoid(gate) * (n @ w["up"].t())) @ w["down"].t() * kept
    z = norm(s, w["last"], w["last_bias"]) @ w["head"].t() + w["head_bias"]
    counts = target.cpu() >= 0
    logp = torch.log_softmax(z, 1)[counts]
    at = target.cpu()[counts]
    loss = (-(1 - model.smoothing) * logp.gather(1, at[:, None])[:, 0] - model.smoothing * logp.mean(1)).mean()
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in w.items()}, x.grad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients(dtype):
    """Norm-wise: a chain of roundings adds up to at most their number times half a step.  fp32: the reductions in the chain
    are at most 2 (2 width + 2 hidden + classes + rows) terms long in all, times 4 for what the norms make of an error
    (|1/std| of these rows is near 1).  bf16: 14 results rounded between x and the farthest gradient and back, 2^-8 each
    and independent, times the same 4."""
    device = torch.device(DEV)
    model = C.Classifier(WIDTH, HIDDEN, CLASSES, device, dtype=dtype, drop=0.25, seed=3)
    g = torch.Generator(device=device).manual_seed(5)
    x, target = C.batch(torch.randn((CLASSES, WIDTH), generator=g, device=device), ROWS, g)
    draw = torch.tensor([99, 7], device=device)
    loss, grads, dx = model.gradients(x.to(dtype), target, draw)
    want_loss, want, want_dx = gradients64(model, x.to(dtype), target, 99, 7)
    tol = (2 * (2 * WIDTH + 2 * HIDDEN + CLASSES + ROWS) * 2.0 ** -24 if dtype is torch.float32 else 14 ** 0.5 * 2.0 ** -8) * 4
    assert abs(float(loss) - float(want_loss)) <= tol * float(want_loss)
    for name, ref in dict(want, x=want_dx).items():
        got = (dx if name == "x" else grads[name]).cpu().double()
        assert float((got - ref).norm()) <= tol * float(ref.norm()), name
    assert not (mic.dropout(torch.ones_like(x), 0.25, draw).cpu().bool()
                ^ torch.from_numpy(T.lots(x.numel(), 99, 7) >= 16384).reshape(x.shape)).any()


def test_captured_steps_are_the_eager_ones():
    """Every replay: the batch it was given, masks of its own step, the eager call's bits."""
    device = torch.device(DEV)
    model = C.Classifier(WIDTH, HIDDEN, CLASSES, device, seed=4)
    step = C.Step(model, ROWS, WIDTH, device)
    g = torch.Generator(device=device).manual_seed(6)
    centres = torch.randn((CLASSES, WIDTH), generator=g, device=device)
    seen = []
    for i in range(4):
        x, target = C.batch(centres, ROWS, g)
        loss, grads = step(x, target)
        torch.cuda.synchronize()
        want_loss, want, want_dx = model.gradients(x.to(torch.bfloat16), target, torch.tensor([1234, i + 1], device=device))
        assert torch.equal(loss, want_loss) and torch.equal(step.dx, want_dx)
        for k in want:
            assert torch.equal(grads[k], want[k]), k
        seen.append(float(loss))
        model.update(grads, 0.01)
    assert len(set(seen)) == 4


def test_it_runs():
    losses = C.main(["--width", "128", "--hidden", "256", "--classes", "500", "--rows", "96", "--steps", "3"])
    assert len(losses) == 3 and all(v == v and abs(v) < 1e9 for v in losses)
