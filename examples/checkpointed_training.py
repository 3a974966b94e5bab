"""A small network trained with 8-bit activation checkpoints and sparsified gradients.

Layers of (1x1 convolution, group normalisation, SiLU) on channels-last
images.  The forward pass keeps, of each layer, its input and the
normalisation's input as 8-bit checkpoints and drops the activations; the
backward pass works from the checkpoints alone and writes every gradient into
its slice of one flat buffer, which the library then sparsifies (error
compensation, top 1 % of each layer) and applies.

    python examples/checkpointed_training.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from layer_wise_top_amd import lags  # noqa: E402

DEV = "cuda"


class Parameters:
    """Weights, gradient and residual of all layers, each one flat fp32 buffer."""

    def __init__(self, shapes, seed=0):
        sizes = [torch.Size(s).numel() for s in shapes]
        self.off = [0]
        for n in sizes:
            self.off.append(self.off[-1] + n)
        self.shapes = shapes
        self.weights = torch.empty(self.off[-1], device=DEV)
        self.grad = torch.zeros_like(self.weights)
        self.residual = torch.zeros_like(self.weights)
        g = torch.Generator(device=DEV).manual_seed(seed)
        for i, s in enumerate(shapes):
            if len(s) == 2:
                w = torch.randn(s, generator=g, device=DEV) / s[1] ** 0.5
            else:                       # gamma and beta, alternating
                w = torch.ones(s, device=DEV) if i % 3 == 1 else torch.zeros(s, device=DEV)
            self.view(self.weights, i).copy_(w)

    def view(self, buf, i):
        return buf[self.off[i]:self.off[i + 1]].view(self.shapes[i])


class Layer:
    """y = silu(groupnorm(x W^T)); parameters first, first + 1, first + 2 of `par`: W, gamma, beta."""

    def __init__(self, par, first, samples, positions, groups, dtype):
        outs, cols = par.shapes[first]
        rows = samples * positions
        self.par, self.first = par, first
        self.gn = lags.GroupNorm(samples, positions, outs, groups, dtype=dtype, act="silu")
        self.gn_ws = lags.gn_workspace(self.gn)
        self.w_ws = lags.wgrad_workspace(rows, outs, cols, dtype)
        self.x8, self.h8 = lags.checkpoint(rows, cols), lags.checkpoint(rows, outs)
        self.mean = torch.empty(samples, groups, device=DEV)
        self.rstd = torch.empty_like(self.mean)

    def _of(self, buf):
        return [self.par.view(buf, self.first + i) for i in range(3)]

    def forward(self, x):
        w, gamma, beta = self._of(self.par.weights)
        lags.lags_ckpt_pack(x, self.x8)
        h = x @ w.to(x.dtype).t()
        lags.lags_gn_forward(self.gn, h, gamma, beta, h, self.mean, self.rstd, self.gn_ws, ckpt=self.h8)
        return h

    def backward(self, dy, need_dx=True):
        w, gamma, beta = self._of(self.par.weights)
        dw, dgamma, dbeta = self._of(self.par.grad)
        lags.lags_gn_backward(self.gn, dy, gamma, beta, self.mean, self.rstd, dy, dgamma, dbeta, self.gn_ws,
                              ckpt=self.h8)
        lags.lags_ckpt_wgrad(dy, self.x8, dw, self.w_ws)
        return dy @ w.to(dy.dtype) if need_dx else None


class Network:
    def __init__(self, samples=32, positions=64, widths=(32, 64, 64, 128), classes=10, groups=8,
                 dtype=torch.bfloat16, seed=0):
        shapes = []
        for cols, outs in zip(widths, widths[1:]):
            shapes += [(outs, cols), (outs,), (outs,)]
        shapes.append((classes, widths[-1]))
        self.par = Parameters(shapes, seed)
        self.layers = [Layer(self.par, 3 * i, samples, positions, groups, dtype) for i in range(len(widths) - 1)]
        self.head = len(shapes) - 1

    def step(self, x, labels):
        """Loss; the gradient of every parameter is left in par.grad."""
        y = x
        for layer in self.layers:
            y = layer.forward(y)
        pooled = y.float().mean(dim=1)
        head = self.par.view(self.par.weights, self.head)
        logp = torch.log_softmax(pooled @ head.t(), dim=1)
        loss = -logp.gather(1, labels[:, None]).mean()
        dlogits = logp.exp()
        dlogits[torch.arange(len(labels), device=DEV), labels] -= 1
        dlogits /= len(labels)
        self.par.view(self.par.grad, self.head).copy_(dlogits.t() @ pooled)
        dy = ((dlogits @ head) / y.shape[1])[:, None, :].expand_as(y).to(y.dtype).contiguous()
        for i in reversed(range(len(self.layers))):
            dy = self.layers[i].backward(dy, need_dx=i > 0)
        return loss


def batch(samples, positions, channels, classes, seed, dtype):
    """Images whose class is the strongest of `classes` fixed patterns in them."""
    fixed = torch.Generator(device=DEV).manual_seed(1234)
    patterns = torch.randn(classes, channels, generator=fixed, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    labels = torch.randint(classes, (samples,), generator=g, device=DEV)
    x = torch.randn(samples, positions, channels, generator=g, device=DEV) + 0.7 * patterns[labels][:, None, :]
    return x.to(dtype), labels


def train(steps=60, lr=0.5, samples=32, positions=64, widths=(32, 64, 64, 128), classes=10,
          dtype=torch.bfloat16, ratio=(1, 100)):
    net = Network(samples, positions, widths, classes, dtype=dtype)
    par = net.par
    layout = lags.Layout(par.off, lags.k_table(par.off, *ratio))
    ws = lags.workspace(layout, 1)
    idx = torch.empty(1, layout.K, dtype=torch.int32, device=DEV)
    val = torch.empty(1, layout.K, device=DEV)
    losses = []
    for i in range(steps):
        x, labels = batch(samples, positions, widths[0], classes, i, dtype)
        losses.append(net.step(x, labels))
        lags.lags_sparsify_layers(layout, par.grad, par.residual, idx[0], val[0], ws)
        lags.lags_aggregate_apply(layout, par.weights, idx, val, 1, lr, ws)
    return [float(v) for v in losses], net


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 200
    losses, net = train(steps)
    kept = sum(layer.x8.numel() + layer.h8.numel() for layer in net.layers)
    rows = net.layers[0].gn.rows
    plain = sum(2 * rows * sum(net.par.shapes[layer.first]) for layer in net.layers)
    for i in range(0, steps, max(1, steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {steps - 1:4d}  loss {losses[-1]:.4f}")
    print(f"activations kept for the backward pass: {kept} bytes (in bf16: {plain})")


if __name__ == "__main__":
    main()
