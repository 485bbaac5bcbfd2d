"""Trains a small stack of pre-norm FFF blocks on one GPU with the library's
own operators: every block is

    h = rms_norm(stream);   y = FFF(h);   stream = stream + y

with the residual's addition done by the next norm.  The step's operators are
rms_norm, forward, backward, rms_norm_backward, grad_norm and adamw_step; torch
holds the tensors and computes the loss.  Weights are bf16 with float32
masters, gradients float32, the residual stream float32, the optimiser's state
float32 or 8 bits.

    python examples/train_block.py --steps 60 --bits 8

With --layer gated the blocks have the dense layer in the FFF layer's place,

    y = (silu(h . W_gate) * (h . W_up)) . W_down

by gated and linear, and everything that its backward pass needs (h, and the
sums of both projections) is kept in 8 bits; the product's own output is made
again from them.

The task is synthetic: targets are a fixed random function of the inputs.
Prints the loss and the gradient's norm; returns them from train().
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_tree_structured_amd as fff  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Model:
    """Parameters by name, with a float32 master and a gradient of each."""

    def __init__(self, layers, d, P, D, h, device, gen, layer="fff"):
        N = 2 ** (D + 1) - 1
        self.layers, self.kind = layers, layer
        init = {}
        for i in range(layers):
            init[f"{i}.gain"] = torch.ones(d)
            if layer == "gated":  # P * h wide
                for k in ("W_gate", "W_up"):
                    init[f"{i}.{k}"] = torch.randn(d, P * h, generator=gen) / math.sqrt(d)
                init[f"{i}.W_down"] = torch.randn(P * h, d, generator=gen) / math.sqrt(P * h)
                continue
            init[f"{i}.W_node"] = torch.randn(P, N, d, generator=gen) / math.sqrt(d)
            init[f"{i}.b_node"] = 0.1 * torch.randn(P, N, generator=gen)
            init[f"{i}.V_node"] = torch.randn(P, N, h, generator=gen) / math.sqrt(h)
            init[f"{i}.W_out"] = torch.randn(P * h, d, generator=gen) / math.sqrt(P * h)
        init["gain"] = torch.ones(d)
        self.master = {k: v.to(device) for k, v in init.items()}
        self.weight = {k: v.to(BF16) for k, v in self.master.items()}
        self.grad = {k: torch.zeros_like(v) for k, v in self.master.items()}

    def layer(self, i):
        return [self.weight[f"{i}.{k}"] for k in ("W_node", "b_node", "V_node", "W_out")]

    def dense(self, i):
        return [self.weight[f"{i}.{k}"] for k in ("W_gate", "W_up", "W_down")]

    def forward(self, stream):
        """The output, and what the backward pass needs of each block."""
        saved, y = [], None
        for i in range(self.layers + 1):
            gain = self.weight[f"{i}.gain"] if i < self.layers else self.weight["gain"]
            if y is None:
                n = fff.rms_norm(stream, gain, want_rstd=True)
            else:
                n = fff.rms_norm(y, gain, residual=stream, want_rstd=True)
                stream = n.residual_out
            if i < self.layers and self.kind == "gated":
                gate, up, down = self.dense(i)
                g = fff.gated(n.y, gate, up, save="e4m3")
                saved.append((stream, n.rstd, (fff.checkpoint(n.y), g.gate, g.up)))
                y = fff.linear(g.h, down).y
                continue
            saved.append((stream, n.rstd, n.y))
            if i == self.layers:
                return n.y, saved
            y, _ = fff.forward(n.y, *self.layer(i), want_path=False)

    def backward(self, dout, saved):
        """Fills every gradient; returns the gradient of the input stream."""
        stream, rstd, _ = saved[self.layers]
        g = fff.rms_norm_backward(dout, stream, self.weight["gain"], rstd, dweight=self.grad["gain"])
        for i in reversed(range(self.layers)):
            stream, rstd, h = saved[i]
            if self.kind == "gated":
                dx = self.dense_backward(i, g.dx, *h)
                g = fff.rms_norm_backward(dx, stream, self.weight[f"{i}.gain"], rstd, dresidual=g.dz,
                                          dweight=self.grad[f"{i}.gain"])
                continue
            out = {f"d{k}": self.grad[f"{i}.{k}"] for k in ("W_node", "b_node", "V_node", "W_out")}
            out["dx"] = torch.empty_like(h)
            fff.backward(h, *self.layer(i), g.dx, out=out)
            g = fff.rms_norm_backward(out["dx"], stream, self.weight[f"{i}.gain"], rstd,
                                      dresidual=g.dz, dweight=self.grad[f"{i}.gain"])
        return g.dz

    def dense_backward(self, i, dy, h, gate, up):
        """The dense layer's gradients from dy and what forward kept."""
        w_gate, w_up, w_down = self.dense(i)
        dprod = fff.linear_backward(dy, None, w_down, want_dW=False).dx
        o = fff.gated_backward(dprod, h, w_gate, w_up, gate, up, want_h=True,
                               dW_gate=self.grad[f"{i}.W_gate"], dW_up=self.grad[f"{i}.W_up"])
        fff.linear_backward(dy, o.h, w_down, want_dx=False, dW=self.grad[f"{i}.W_down"])
        return o.dx

    def optimiser(self, bits, weight_decay):
        """The optimiser's table (matrices decay, gains and biases do not)."""
        names = list(self.weight)
        params = [self.weight[k] for k in names]
        m, v, scales = fff.adamw_state(params, bits)
        decay = [weight_decay if self.weight[k].dim() > 1 and "b_node" not in k else 0.0 for k in names]
        return fff.adamw_table(params, [self.grad[k] for k in names], m, v,
                               masters=[self.master[k] for k in names], scales=scales,
                               weight_decay=decay)


def train(steps=60, layers=2, T=512, d=256, P=4, D=3, h=64, bits=8, lr=2e-3, seed=0, device="cuda:0",
          log=None, layer="fff"):
    """[(loss, gradient norm)] of every step."""
    gen = torch.Generator().manual_seed(seed)
    model = Model(layers, d, P, D, h, device, gen, layer)
    stream = torch.randn(T, d, generator=gen).to(device)
    target = torch.tanh(stream @ (torch.randn(d, d, generator=gen) / math.sqrt(d)).to(device))
    table = model.optimiser(bits, weight_decay=0.01)
    history = []
    for step in range(1, steps + 1):
        out, saved = model.forward(stream)
        error = out.float() - target
        model.backward((error * (2.0 / error.numel())).to(BF16), saved)
        norm = fff.grad_norm(table, max_norm=1.0)
        fff.adamw_step(table, lr=lr, step=step, beta2=0.99, grad_scale=norm[1:],
                       seed=seed + step if bits == 8 else None)
        history.append((error.square().mean(), norm[0]))
        if log and (step == 1 or step % 10 == 0):
            log(f"step {step}: loss {float(history[-1][0]):.4f}, gradient norm {float(norm[0]):.4f}")
    return [(float(a), float(b)) for a, b in history]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--bits", type=int, default=8, choices=[8, 32])
    ap.add_argument("--layer", default="fff", choices=["fff", "gated"])
    a = ap.parse_args()
    train(a.steps, a.layers, a.tokens, bits=a.bits, log=print, layer=a.layer)


if __name__ == "__main__":
    main()
