"""The operators together, as the example runs them: a stack of pre-norm FFF
blocks learns, with either state, and its gradients are those of float64
differences along the weights."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_the_example_learns(bits):
    h = np.array(example().train(steps=40, bits=bits))
    assert np.isfinite(h).all()
    assert h[-5:, 0].mean() < 0.7 * h[0, 0]


def test_eight_bit_states_follow_the_exact_ones():
    """The same 40 steps with either state: each update differs by the state's
    rounding (an e4m3 step is at most an eighth of a moment) without a bias,
    so the losses stay within a tenth of the progress made."""
    m = example()
    a, b = (np.array(m.train(steps=40, bits=bits))[:, 0] for bits in (32, 8))
    assert abs(a[-5:].mean() - b[-5:].mean()) < 0.1 * (a[0] - a[-5:].mean())


def gelu(a):
    return 0.5 * a * (1 + np.tanh(np.sqrt(2 / np.pi) * (a + 0.044715 * a ** 3)))


def block_loss(stream, W, target, eps=1e-6):
    """The example's forward pass and loss in float64, on the CPU."""
    s, y = stream, None
    layers = sum(k.endswith(".gain") for k in W)
    for i in range(layers + 1):
        gain = W[f"{i}.gain"] if i < layers else W["gain"]
        s = s if y is None else s + y
        x = s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * gain
        if i == layers:
            return ((x - target) ** 2).mean()
        Wn, b, V, Wo = (W[f"{i}.{k}"] for k in ("W_node", "b_node", "V_node", "W_out"))
        P, N, _ = Wn.shape
        H = np.zeros((len(x), P, V.shape[2]))
        for p in range(P):
            n = np.zeros(len(x), np.int64)
            while True:
                a = (x * Wn[p, n]).sum(1) + b[p, n]
                H[:, p] += gelu(a)[:, None] * V[p, n]
                nxt = 2 * n + 1 + (a >= 0)
                if nxt[0] >= N:
                    break
                n = nxt
        y = H.reshape(len(x), -1) @ Wo


def test_gradients_of_the_stack_against_differences():
    """Every parameter's gradient along its own direction against a float64
    central difference of the whole stack.  The device rounds h, y and the
    weights' products to bf16 (2^-8 each, half a dozen on the way), and those
    errors average over a parameter's elements: 5 % is a wide bound for the
    projection on the gradient itself."""
    m = example()
    gen = torch.Generator().manual_seed(3)
    model = m.Model(2, 64, 2, 2, 32, "cuda:0", gen)
    stream = torch.randn(96, 64, generator=gen).to("cuda:0")
    target = torch.randn(96, 64, generator=gen).to("cuda:0")
    out, saved = model.forward(stream)
    error = out.float() - target
    model.backward((error * (2.0 / error.numel())).to(torch.bfloat16), saved)
    W = {k: v.double().cpu().numpy() for k, v in model.weight.items()}
    s, t = stream.double().cpu().numpy(), target.double().cpu().numpy()
    assert abs(block_loss(s, W, t) - float(error.square().mean())) < 0.02 * block_loss(s, W, t)
    for k, g in model.grad.items():
        g = g.double().cpu().numpy()
        size = np.linalg.norm(g)
        e = g / size
        h = 1e-5  # small enough that hardly a logit changes its sign
        d = (block_loss(s, dict(W, **{k: W[k] + h * e}), t) - block_loss(s, dict(W, **{k: W[k] - h * e}), t)) / (2 * h)
        assert abs(d - size) < 0.05 * size, (k, d, size)
