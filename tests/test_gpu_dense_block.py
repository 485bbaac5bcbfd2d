"""The dense block's operators together, as a training step and a decode step
run them: the norm, the gated pair with its sums kept in 8 bits, the down
projection onto the residual stream, and back."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import dense_oracle as O
import sparse_tree_structured_amd as fff

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV, B, F64 = "cuda:0", torch.bfloat16, torch.float64


def example():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_the_example_runs_with_the_dense_layer(bits):
    print("[gpu] example, gated", bits, flush=True)
    h = np.array(example().train(steps=6, bits=bits, layer="gated"))
    assert h.shape == (6, 2) and np.isfinite(h).all() and (h > 0).all()


def block_loss(stream, W, target, eps=1e-6):
    """The example's forward pass and loss with the dense layer, in float64."""
    s, y = stream, None
    layers = sum(k.endswith(".gain") for k in W)
    for i in range(layers + 1):
        gain = W[f"{i}.gain"] if i < layers else W["gain"]
        s = s if y is None else s + y
        x = s * (s.square().mean(1, keepdim=True) + eps).rsqrt() * gain
        if i == layers:
            return (x - target).square().mean()
        h = O.activation(x @ W[f"{i}.W_gate"], "silu")[0] * (x @ W[f"{i}.W_up"])
        y = h @ W[f"{i}.W_down"]


def test_gradients_of_the_stack_against_differences():
    """Every parameter's gradient along its own direction against a float64
    central difference.  A gradient that is off by a share r of its size in
    other directions is longer by r^2 / 2 and leans by as much, so the two
    differ by r^2.  A value kept in 8 bits is off by at most 2^-4, 1/28 on
    average over a step, and three such values meet in a gradient, with some
    ten roundings to bf16: r is below 0.1, r^2 below 1 %; 5 % is allowed."""
    m = example()
    print("[gpu] gradients of the gated stack", flush=True)
    gen = torch.Generator().manual_seed(3)
    model = m.Model(2, 64, 2, 2, 48, DEV, gen, "gated")
    stream = torch.randn(96, 64, generator=gen).to(DEV)
    target = torch.randn(96, 64, generator=gen).to(DEV)
    out, saved = model.forward(stream)
    error = out.float() - target
    model.backward((error * (2.0 / error.numel())).to(B), saved)
    W = {k: v.to(F64) for k, v in model.weight.items()}
    s, t = stream.to(F64), target.to(F64)
    for k, g in model.grad.items():
        g = g.to(F64)
        size = float(g.norm())
        e = g / size
        d = float(block_loss(s, dict(W, **{k: W[k] + 1e-5 * e}), t) -
                  block_loss(s, dict(W, **{k: W[k] - 1e-5 * e}), t)) / 2e-5
        assert abs(d - size) < 0.05 * size, (k, d, size)


@pytest.mark.parametrize("T,d,F", [(1, 128, 344), (33, 200, 520), (600, 256, 688)])
def test_a_block_forward_and_back(T, d, F):
    """The block's outputs against float64 from the same rounded inputs of
    each operator (their own bounds), eager and captured alike."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T)
    print("[gpu] block", T, d, F, flush=True)

    def rand(*s, size=1.0):
        return size * torch.randn(*s, generator=gen, device=DEV)

    x, r = rand(T, d, size=0.3).to(B), rand(T, d)
    gain, Wg, Wu = rand(d).to(B), rand(d, F, size=d ** -0.5).to(B), rand(d, F, size=d ** -0.5).to(B)
    Wd, dy = rand(F, d, size=F ** -0.5).to(B), rand(T, d).to(B)

    def step():
        n = fff.rms_norm(x, gain, residual=r, want_rstd=True)
        kept = fff.checkpoint(n.y, 32)
        g = fff.gated(n.y, Wg, Wu, save="e4m3", group=64)
        y = fff.linear(g.h, Wd, residual=n.residual_out).y
        dh = fff.linear_backward(dy, None, Wd, want_dW=False).dx
        b = fff.gated_backward(dh, kept, Wg, Wu, g.gate, g.up, want_h=True, grad_dtype=B)
        dWd = fff.linear_backward(dy, b.h, Wd, want_dx=False).dW
        z = fff.rms_norm_backward(b.dx, n.residual_out, gain, n.rstd, dresidual=None)
        return dict(n=n.y, z=n.residual_out, h=g.h, y=y, dh=dh, dx=b.dx, dWg=b.dW_gate, dWu=b.dW_up, h2=b.h,
                    dWd=dWd, dz=z.dz, dgain=z.dweight, kept=kept, gate=g.gate, up=g.up)

    o = step()
    torch.cuda.synchronize()
    u = O.U["bf16"]
    w = {k: v.to(F64) for k, v in dict(Wg=Wg, Wu=Wu, Wd=Wd).items()}
    _, _, _, _, h, eh = O.gated(o["n"].to(F64), w["Wg"], w["Wu"], "silu")
    O.close(o["h"], h, eh + (h.abs() + eh) * u, "h")
    y, ey = O.product(o["h"].to(F64), w["Wd"])
    assert o["y"].dtype is torch.float32
    O.close(o["y"], y + o["z"].to(F64), ey + (y + o["z"].to(F64)).abs() * 2 * O.U32, "y")
    dh, e = O.product(dy.to(F64), w["Wd"].t())
    O.close(o["dh"], dh, e + (dh.abs() + e) * u, "dh")
    g, up = (O.load(o[k].codes, o[k].scale, 64) for k in ("gate", "up"))
    value, slope, ev, es = O.activation(g, "silu")
    O.close(o["h2"], value * up, ev * up.abs() + (value * up).abs() * (u + 4 * O.U32) + O.FLOOR, "h made again")
    dhv = o["dh"].to(F64)
    dg, du = dhv * up * slope, dhv * value
    eg = (dhv * up).abs() * es + dg.abs() * (u + 4 * O.U32)
    eu = dhv.abs() * ev + du.abs() * (u + 4 * O.U32)
    dx, ex = O.product(torch.cat([dg, du], 1), torch.cat([w["Wg"], w["Wu"]], 1).t(), torch.cat([eg, eu], 1))
    O.close(o["dx"], dx, ex + (dx.abs() + ex) * u, "dx")
    xv = O.load(o["kept"].codes, o["kept"].scale, 32)
    dWg, ew = O.product(xv.t(), dg, xv.t().abs() * u, eg)
    O.close(o["dWg"], dWg, ew + (dWg.abs() + ew) * u, "dWg")
    dWd, ew = O.product(o["h2"].to(F64).t(), dy.to(F64))
    O.close(o["dWd"], dWd, ew + dWd.abs() * O.U32, "dWd")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        again = step()
        torch.cuda.synchronize()
        for k in ("y", "h", "dx", "dWg", "dWu", "dWd", "dz", "dgain"):
            assert torch.equal(captured[k], again[k]) and torch.equal(again[k], o[k]), k


def test_decode_steps_through_one_layer():
    """Tokens one by one give what the batch gives, within both sides' bounds."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    print("[gpu] decode steps", flush=True)
    T, d, F = 40, 256, 1024
    x, Wg, Wu, Wd = ((torch.randn(*s, generator=gen, device=DEV) * k).to(B) for s, k in
                     (((T, d), 1.0), ((d, F), d ** -0.5), ((d, F), d ** -0.5), ((F, d), F ** -0.5)))
    stream = torch.randn(T, d, generator=gen, device=DEV)
    h = torch.cat([fff.gated(x[i:i + 1], Wg, Wu).h for i in range(T)])
    y = torch.cat([fff.linear(h[i:i + 1], Wd, residual=stream[i:i + 1]).y for i in range(T)])
    *_, want, eh = O.gated(x.to(F64), Wg.to(F64), Wu.to(F64), "silu")
    O.close(h, want, eh + (want.abs() + eh) * O.U["bf16"], "h")
    want, ey = O.product(h.to(F64), Wd.to(F64))
    want = want + stream.to(F64)
    O.close(y, want, ey + want.abs() * 2 * O.U32, "y")
    batch = fff.linear(h, Wd, residual=stream).y
    O.close(batch, want, ey + want.abs() * 2 * O.U32, "the batch")
