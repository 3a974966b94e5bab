"""The example that runs the activation operators and the sparsified update together."""
import importlib.util
import os

import numpy as np
import pytest

import act_reference as R

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "checkpointed_training.py")


def _module():
    spec = importlib.util.spec_from_file_location("checkpointed_training", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_the_loss():
    """Ten classes from 5 % of each layer's entries a step: from about log 10 to less than half."""
    losses, _ = _module().train(steps=120, ratio=(1, 20))
    print("loss", losses[0], "->", np.mean(losses[-10:]), flush=True)
    assert np.isfinite(losses).all()
    assert np.mean(losses[-10:]) < 0.5 * np.mean(losses[:3])


def test_step_against_float64():
    """One fp32 step's gradients against float64 with the checkpoints' values in the backward pass.
    What differs: fp32 sums of up to 512 terms through three layers (about 1e-6), and codes that
    round the other way because the value they stand for came out of such sums: one in about 1e5
    moves by a step, 1/64 of its run's largest value, which is 1/64 * sqrt(1e-5) = 5e-5 of a
    gradient's norm.  1e-3 is twenty times that."""
    import torch
    m = _module()
    net = m.Network(samples=8, positions=64, dtype=torch.float32, seed=3)
    par = net.par
    x, labels = m.batch(8, 64, 32, 10, 5, torch.float32)
    net.step(x, labels)
    torch.cuda.synchronize()
    W = [par.view(par.weights, i).double().cpu().numpy() for i in range(len(par.shapes))]
    y, kept = x.double().cpu().numpy(), []
    for i in range(3):
        w, ga, be = W[3 * i:3 * i + 3]
        h = y @ w.T
        x8 = R.held(y.reshape(-1, y.shape[2]))
        h8 = R.held(h.reshape(-1, h.shape[2])).reshape(h.shape)
        mean, rstd = R.stats(h, 8, 1e-5)
        kept.append((x8, h8, mean, rstd))
        c = h.shape[2]
        y = R.act((h - R.per_channel(mean, c)) * R.per_channel(rstd, c) * ga + be, "silu")
    pooled, lab = y.mean(axis=1), labels.cpu().numpy()
    z = pooled @ W[9].T
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    p[np.arange(8), lab] -= 1
    p /= 8
    want = {9: p.T @ pooled}
    dy = np.broadcast_to(((p @ W[9]) / 64)[:, None, :], y.shape)
    for i in (2, 1, 0):
        x8, h8, mean, rstd = kept[i]
        (dh, want[3 * i + 1], want[3 * i + 2]), _ = R.backward(dy, h8, W[3 * i + 1], W[3 * i + 2], mean, rstd, "silu")
        want[3 * i] = dh.reshape(-1, dh.shape[2]).T @ x8
        dy = dh @ W[3 * i]
    for i, w in want.items():
        got = par.view(par.grad, i).double().cpu().numpy()
        err = np.linalg.norm(got - w) / np.linalg.norm(w)
        print("parameter", i, "relative error", err, flush=True)
        assert err < 1e-3, i
