"""Plain float64 forms of the dense feed-forward operators with bounds on what
32-bit sums and one rounding of each operand and output can change.  Written
from the formulas, apart from the kernels; torch in float64 on any device.

Bounds.  A sum of n products in 32 bits, in any order, is off by at most
(n + 8) 2^-24 of the sum of their sizes; twice that is allowed, for matrix
cores that do not round each step to nearest.  An activation's logistic
function of z is off by (4 |z| + 8) 2^-24 of itself (z's own four roundings,
the exponent's one, and the last three), its product with two more factors by
a few units more: (6 |z| + 16) 2^-24.  What is below 2^-120 counts for nothing.
A rounding to a type is off by u of the value."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
U32 = 2.0 ** -24
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TY = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
TINY = 2.0 ** -126
FLOOR = 2.0 ** -120
K2 = 2.0 * math.sqrt(2.0 / math.pi)


def sum_u(n):
    return (n + 8) * 2.0 ** -23


def logit(a, act):
    return K2 * (a + 0.044715 * a ** 3) if act == "gelu" else a


def activation(a, act):
    """(value, derivative, bound of the value's error, bound of the derivative's)."""
    if act == "none":
        return a, torch.ones_like(a), torch.zeros_like(a), torch.zeros_like(a)
    if act == "relu":
        on = (a > 0).to(F64)
        return torch.where(a > 0, a, torch.zeros_like(a)), on, torch.zeros_like(a), torch.zeros_like(a)
    z = logit(a, act)
    q = torch.sigmoid(z)
    p = torch.sigmoid(-z)  # 1 - q without cancellation
    dz = K2 * (1 + 3 * 0.044715 * a ** 2) if act == "gelu" else torch.ones_like(a)
    value, tail = a * q, a * q * p * dz
    off = (6 * z.abs() + 16) * U32
    # (1 - q in 32 bits is off by the rounding of q as well)
    return value, q + tail, value.abs() * off + FLOOR, q * off + tail.abs() * off + (value * dz).abs() * (2 * U32 + q * off) + FLOOR


# The largest slope of an activation (GELU 1.129, SiLU 1.0998).
SLOPE = 1.13


def product(a, b, ea=None, eb=None):
    """a @ b in float64 and the bound of its error in 32 bits, where a and b
    are off by ea and eb."""
    n = a.shape[1]
    size = a.abs() @ b.abs()
    err = sum_u(n) * size
    if ea is not None:
        err = err + ea @ b.abs()
    if eb is not None:
        err = err + a.abs() @ eb
    return a @ b, err


def linear(x, W, bias, residual, act):
    """(a, bound, y, bound before y's rounding)."""
    a, err = product(x, W)
    if bias is not None:
        a, err = a + bias, err + (a + bias).abs() * U32
    value, _, off, _ = activation(a, act)
    y, ey = value, off * 1.01 + SLOPE * err
    if residual is not None:
        y = y + residual
        ey = ey + y.abs() * U32
    return a, err, y, ey


def gated(x, Wg, Wu, act):
    (g, eg), (u, eu) = product(x, Wg), product(x, Wu)
    value, _, off, _ = activation(g, act)
    ev = off * 1.01 + SLOPE * eg
    return g, eg, u, eu, value * u, ev * (u.abs() + eu) + value.abs() * eu + (value * u).abs() * U32


def close(got, want, bound, what):
    got = got.to(F64)
    err = (got - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), \
        f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((err - bound)[bad].max()):.3g}, " \
        f"first at {bad.nonzero()[0].tolist()}"


def group_amax(a, group):
    T, d = a.shape
    g = group or d
    return torch.nn.functional.pad(a.abs(), (0, -d % g)).view(T, -1, g).amax(2)


def spread(scale, group, d):
    """A scale for every column."""
    return scale.repeat_interleave(group or d, 1)[:, :d]


def load(codes, scale, group):
    """The values of a checkpoint, in 32 bits, as float64."""
    return (codes.float() * spread(scale, group, codes.shape[1])).to(F64)


def nearest(t):
    """t (float64, at most 448) as e4m3 values.  The conversion goes by way of
    float32: one rounding more, which moves t by 2^-24 of itself."""
    return t.clamp(-448.0, 448.0).float().to(F8).to(F64)


def check_checkpoint(kept, a, err, group, what):
    """Scales of the groups' largest sizes, and codes between those of the
    ends of what a value can be."""
    want = (group_amax(a, group) / 448).clamp(min=TINY)
    off = group_amax(err, group) / 448 + want * 4 * U32
    close(kept.scale, want, off, f"{what}'s scales")
    s = spread(kept.scale.to(F64), group, a.shape[1])
    lo, hi = (a - err) / s, (a + err) / s
    lo, hi = lo - lo.abs() * 8 * U32, hi + hi.abs() * 8 * U32
    got = kept.codes.to(F64)
    assert bool(((got >= nearest(lo)) & (got <= nearest(hi))).all()), f"{what}'s codes"
