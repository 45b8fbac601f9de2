"""A classifier over a large number of classes, trained with the library's operators.

    python examples/classifier.py [--width 4096 --hidden 9216 --classes 50021 --rows 4096 --steps 10]

One feed-forward sublayer and a head:

    n = layer_norm(x)                    h = silu(W_gate n) * (W_up n)
    s = x + dropout(W_down h)            y = layer_norm(s)
    loss = cross entropy of softmax(W_head y + b_head), labels smoothed, rows without a class left out

Neither dropout's masks nor the logits are kept.  Forward and gradients are
captured into one graph; a seed and a step number in device memory make every
replay draw masks of its own.  Weights train in bf16 beside fp32 ones.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import convolution_forward_conv2d_amd as mic  # noqa: E402

IGNORED = -100


class Classifier:
    def __init__(self, width, hidden, classes, device, dtype=torch.bfloat16, drop=0.1, smoothing=0.1, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def matrix(rows, cols):
            return torch.randn((rows, cols), generator=g, device=device).mul_(cols ** -0.5)

        def ones():
            return torch.ones(width, device=device)

        def zeros(n=width):
            return torch.zeros(n, device=device)

        self.master = {"norm": ones(), "norm_bias": zeros(), "gate": matrix(hidden, width), "up": matrix(hidden, width),
                       "down": matrix(width, hidden), "last": ones(), "last_bias": zeros(), "head": matrix(classes, width),
                       "head_bias": zeros(classes)}
        self.momentum = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.w = {k: v.to(dtype) for k, v in self.master.items()}
        self.drop, self.smoothing = drop, smoothing

    def gradients(self, x, target, draw):
        """(loss, gradients of the weights, gradient of x); draw: the seed and the step, int64 on the device."""
        w = self.w
        n = mic.layer_norm(x, w["norm"], bias=w["norm_bias"])
        h, gate, up = mic.gated_linear(n.y, w["gate"], w["up"], return_products=True)
        s = mic.dropout(mic.linear(h, w["down"]), self.drop, draw, residual=x)
        y = mic.layer_norm(s, w["last"], bias=w["last_bias"])
        r = mic.linear_cross_entropy(y.y, w["head"], target, bias=w["head_bias"], ignore_index=IGNORED,
                                     label_smoothing=self.smoothing)

        one = torch.ones_like(r.loss)
        g = {}
        dy, g["head"], g["head_bias"] = mic.linear_cross_entropy_backward(
            one, y.y, w["head"], target, r.lse, bias=w["head_bias"], count=r.count, ignore_index=IGNORED,
            label_smoothing=self.smoothing)
        ds, g["last"], g["last_bias"] = mic.layer_norm_backward(dy, y.sum, w["last"], y.mean, y.rstd, bias=True)
        dout = mic.dropout_backward(ds, self.drop, draw)
        dh, g["down"], _ = mic.linear_backward(dout, h, w["down"])
        dn, g["gate"], g["up"] = mic.gated_linear_backward(dh, n.y, w["gate"], w["up"], gate, up)
        dx, g["norm"], g["norm_bias"] = mic.layer_norm_backward(dn, n.sum, w["norm"], n.mean, n.rstd, dsum=ds, bias=True)
        return r.loss, g, dx

    def update(self, grads, rate, keep=0.9):
        for k, v in self.master.items():
            self.momentum[k].mul_(keep).add_(grads[k].float())
            v.add_(self.momentum[k], alpha=-rate)
            self.w[k].copy_(v)


class Step:
    """Forward and gradients of one batch in a graph."""

    def __init__(self, model, rows, width, device):
        self.x = torch.zeros((rows, width), dtype=model.w["norm"].dtype, device=device)
        self.target = torch.zeros(rows, dtype=torch.int64, device=device)
        self.draw = torch.tensor([1234, 0], device=device)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            model.gradients(self.x, self.target, self.draw)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.loss, self.grads, self.dx = model.gradients(self.x, self.target, self.draw)

    def __call__(self, x, target):
        self.x.copy_(x)
        self.target.copy_(target)
        self.draw[1] += 1
        self.graph.replay()
        return self.loss, self.grads


def batch(centres, rows, g):
    """Rows around the centres of their classes, the last sixteenth padding."""
    target = torch.randint(0, centres.shape[0], (rows,), generator=g, device=centres.device)
    x = centres[target] + 0.5 * torch.randn((rows, centres.shape[1]), generator=g, device=centres.device)
    target[rows - rows // 16:] = IGNORED
    return x, target


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=9216)
    p.add_argument("--classes", type=int, default=50021)
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--steps", type=int, default=10)
    p.add_argument("--rate", type=float, default=0.05)
    a = p.parse_args(argv)
    device = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=device).manual_seed(1)
    centres = torch.randn((a.classes, a.width), generator=g, device=device)
    model = Classifier(a.width, a.hidden, a.classes, device)
    step = Step(model, a.rows, a.width, device)
    losses, seconds = [], 0.0
    for _ in range(a.steps):
        x, target = batch(centres, a.rows, g)
        torch.cuda.synchronize()
        start = time.perf_counter()
        loss, grads = step(x, target)
        torch.cuda.synchronize()
        seconds += time.perf_counter() - start
        losses.append(float(loss))
        model.update(grads, a.rate)
    print("loss %.4f -> %.4f in %d steps, %.2f ms for a batch's loss and gradients" % (losses[0], losses[-1], a.steps,
                                                                                      seconds / a.steps * 1e3))
    return losses


if __name__ == "__main__":
    main()
