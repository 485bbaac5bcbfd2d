"""The dense feed-forward operators on the GPU against their float64 forms
(dense_oracle.py, which derives the bounds)."""
import math
import zlib

import pytest
import torch

import dense_oracle as O
import sparse_tree_structured_amd as fff

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TY, U, F64 = O.TY, O.U, O.F64
NAME = {torch.float32: "f32", torch.bfloat16: "bf16"}


def randn(gen, *shape, ty="f32", size=1.0):
    return (size * torch.randn(*shape, generator=gen, device=DEV)).to(TY[ty])


def seeded(*key):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(zlib.crc32(repr(key).encode()))
    return gen


def say(*what):
    print("[gpu]", *what, flush=True)


def d64(t):
    return None if t is None else t.to(F64)


def check_saved(kept, a, err, save, group, ty, what):
    if save is None:
        assert kept is None
    elif save == "same":
        assert kept.dtype is TY[ty]
        O.close(kept, a, err + (a.abs() + err) * U[ty], what)
    else:
        assert kept.group == group
        O.check_checkpoint(kept, a, err, group, what)


def check_linear(T, K, N, ty, out, act="none", bias=False, residual=False, save=None, group=128, seed=0,
                 **kw):
    gen = seeded(T, K, N, seed)
    say("linear", T, K, N, ty, out, act, bias, residual, save, group)
    x, W = randn(gen, T, K, ty=ty), randn(gen, K, N, ty=ty, size=1 / math.sqrt(K))
    b = randn(gen, N, ty=ty) if bias else None
    r = randn(gen, T, N, ty=out, size=2.0) if residual else None
    o = fff.linear(x, W, b, residual=r, act=act, out_dtype=TY[out], save=save, group=group, **kw)
    torch.cuda.synchronize()
    a, err, y, ey = O.linear(d64(x), d64(W), d64(b), d64(r), act)
    assert o.y.dtype is TY[out]
    O.close(o.y, y, ey + (y.abs() + ey) * U[out], "y")
    check_saved(o.pre, a, err, save, group, ty, "pre")
    return o


def check_gated(T, K, N, ty, act="silu", save=None, group=128, seed=0):
    gen = seeded(T, K, N, seed)
    say("gated", T, K, N, ty, act, save, group)
    x = randn(gen, T, K, ty=ty)
    Wg, Wu = (randn(gen, K, N, ty=ty, size=1 / math.sqrt(K)) for _ in range(2))
    o = fff.gated(x, Wg, Wu, act=act, save=save, group=group)
    torch.cuda.synchronize()
    g, eg, u, eu, h, eh = O.gated(d64(x), d64(Wg), d64(Wu), act)
    O.close(o.h, h, eh + (h.abs() + eh) * U[ty], "h")
    check_saved(o.gate, g, eg, save, group, ty, "gate")
    check_saved(o.up, u, eu, save, group, ty, "up")
    return o


def keep(x, ty, group):
    """x as it is kept (group None: in the layer's type), and its values."""
    if group is None:
        x = x.to(TY[ty])
        return x, x.to(F64)
    c = fff.checkpoint(x.to(TY[ty]), group)
    return c, O.load(c.codes, c.scale, group)


def as_operand(v, ty, eight):
    """The bound of a value's rounding to the layer's type."""
    return v.abs() * U[ty] if eight and ty == "bf16" else None


def check_linear_back(T, K, N, ty, act="none", group=None, x_group=None, grad="f32", bias=True, seed=0):
    gen = seeded(T, K, N, seed)
    say("linear backward", T, K, N, ty, act, group, x_group, grad)
    dy, W = randn(gen, T, N, ty=ty), randn(gen, K, N, ty=ty, size=1 / math.sqrt(K))
    x, xv = keep(randn(gen, T, K), ty, x_group)
    pre, pv = keep(randn(gen, T, N, size=2.0), ty, group) if act != "none" else (None, None)
    o = fff.linear_backward(dy, x, W, act=act, pre=pre, want_dbias=bias, grad_dtype=TY[grad])
    torch.cuda.synchronize()
    da, e = d64(dy), None
    if act != "none":
        _, slope, _, off = O.activation(pv, act)
        e32 = da.abs() * off + (da * slope).abs() * 2 * O.U32
        da = da * slope
        e = e32 + (da.abs() + e32) * U[ty]
    else:
        e32 = torch.zeros_like(da)
    dx, ex = O.product(da, d64(W).t(), e)
    O.close(o.dx, dx, ex + (dx.abs() + ex) * U[ty], "dx")
    dW, ew = O.product(xv.t(), da, as_operand(xv.t(), ty, x_group is not None), e)
    O.close(o.dW, dW, ew + (dW.abs() + ew) * U[grad], "dW")
    if bias:
        O.close(o.dbias, da.sum(0), O.sum_u(T) * da.abs().sum(0) + e32.sum(0), "dbias")
    return o


def check_gated_back(T, K, N, ty, act="silu", group=None, x_group=None, grad="f32", want_h=True, seed=0):
    gen = seeded(T, K, N, seed)
    say("gated backward", T, K, N, ty, act, group, x_group, grad)
    dh = randn(gen, T, N, ty=ty)
    Wg, Wu = (randn(gen, K, N, ty=ty, size=1 / math.sqrt(K)) for _ in range(2))
    x, xv = keep(randn(gen, T, K), ty, x_group)
    (gate, g), (up, u) = (keep(randn(gen, T, N, size=2.0), ty, group) for _ in range(2))
    o = fff.gated_backward(dh, x, Wg, Wu, gate, up, act=act, want_h=want_h, grad_dtype=TY[grad])
    torch.cuda.synchronize()
    value, slope, ev, es = O.activation(g, act)
    d = d64(dh)
    dg, du = d * u * slope, d * value
    eg = (d * u).abs() * es + dg.abs() * 3 * O.U32
    eu = d.abs() * ev + du.abs() * 2 * O.U32
    eg, eu = eg + (dg.abs() + eg) * U[ty], eu + (du.abs() + eu) * U[ty]
    dx, ex = O.product(torch.cat([dg, du], 1), torch.cat([d64(Wg), d64(Wu)], 1).t(), torch.cat([eg, eu], 1))
    O.close(o.dx, dx, ex + (dx.abs() + ex) * U[ty], "dx")
    xe = as_operand(xv.t(), ty, x_group is not None)
    for got, da, e, what in ((o.dW_gate, dg, eg, "dW_gate"), (o.dW_up, du, eu, "dW_up")):
        dW, ew = O.product(xv.t(), da, xe, e)
        O.close(got, dW, ew + (dW.abs() + ew) * U[grad], what)
    if want_h:
        eh = ev * u.abs() + (value * u).abs() * 2 * O.U32
        O.close(o.h, value * u, eh + ((value * u).abs() + eh) * U[ty], "h")
    else:
        assert o.h is None
    return o


# Rows around one, the tiles' and the small kernels' edges; widths odd, in
# eights, and around the tiles'.
SIZES = [(1, 1, 1), (1, 64, 64), (2, 7, 5), (1, 33, 129), (3, 100, 255), (5, 767, 130), (16, 256, 256),
         (17, 255, 257), (33, 72, 136), (64, 520, 384), (65, 64, 8), (127, 31, 300), (128, 128, 512),
         (129, 96, 264), (200, 1000, 264), (257, 40, 513), (300, 392, 1000)]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("ty,out", TYPES)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear(T, K, N, ty, out):
    check_linear(T, K, N, ty, out)
    check_linear(T, K, N, ty, out, act="gelu", bias=True, residual=True, seed=1)


@pytest.mark.parametrize("ty,out", TYPES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "relu"])
@pytest.mark.parametrize("T,K,N", [(3, 40, 136), (70, 96, 200), (260, 64, 259)])
def test_linear_saves(T, K, N, act, ty, out):
    check_linear(T, K, N, ty, out, act=act, bias=True, save="same")
    for group in (32, 64, 128):
        check_linear(T, K, N, ty, out, act=act, residual=True, save="e4m3", group=group, seed=group)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_gated(T, K, N, ty):
    check_gated(T, K, N, ty)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "relu"])
@pytest.mark.parametrize("T,K,N", [(1, 64, 136), (70, 96, 200), (260, 64, 259)])
def test_gated_saves(T, K, N, act, ty):
    check_gated(T, K, N, ty, act=act, save="same")
    for group in (32, 64, 128):
        check_gated(T, K, N, ty, act=act, save="e4m3", group=group, seed=group)


@pytest.mark.parametrize("ty,grad", TYPES)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear_backward(T, K, N, ty, grad):
    check_linear_back(T, K, N, ty, grad=grad)
    check_linear_back(T, K, N, ty, act="gelu", group=64, x_group=32, grad=grad, seed=1)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
@pytest.mark.parametrize("group,x_group", [(None, None), (32, None), (128, 0), (0, 128), (None, 64)])
def test_linear_backward_kept(act, group, x_group, ty):
    check_linear_back(70, 96, 200, ty, act=act, group=group, x_group=x_group)


@pytest.mark.parametrize("ty,grad", TYPES)
@pytest.mark.parametrize("T,K,N", SIZES)
def test_gated_backward(T, K, N, ty, grad):
    check_gated_back(T, K, N, ty, grad=grad)
    check_gated_back(T, K, N, ty, act="gelu", group=64, x_group=32, grad=grad, want_h=False, seed=1)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "relu"])
@pytest.mark.parametrize("group,x_group", [(None, None), (32, None), (128, 0), (0, 128), (None, 64)])
def test_gated_backward_kept(act, group, x_group, ty):
    check_gated_back(70, 96, 200, ty, act=act, group=group, x_group=x_group)


# ---- checkpoints: the formula's bits ----

def plain_save(x, group):
    """fff.h's formula in 32 bits, operation by operation."""
    T, d = x.shape
    g = torch.nn.functional.pad(x.float(), (0, -d % (group or d))).view(T, -1, group or d)
    scale = (g.abs().amax(2) * torch.tensor(1 / 448, device=DEV)).clamp(min=O.TINY)
    codes = (g * (1.0 / scale)[:, :, None]).clamp(-448, 448).to(O.F8).view(T, -1)[:, :d]
    return codes, scale


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 30), (5, 129), (64, 768), (2, 2047), (33, 2048), (7, 9001)])
def test_checkpoint(T, d, group, ty):
    gen = seeded(T, d, group)
    say("checkpoint", T, d, group, ty)
    x = randn(gen, T, d, ty=ty) * torch.exp(4 * randn(gen, T, 1)).to(TY[ty])
    x[:, ::7] = 0
    c = fff.checkpoint(x, group)
    codes, scale = plain_save(x, group)
    assert torch.equal(c.scale, scale)
    assert torch.equal(c.codes.float(), codes.float())
    for out in ("f32", "bf16"):
        r = fff.restore(c, TY[out])
        want = codes.float() * O.spread(scale, group, d)
        assert torch.equal(r, want.to(TY[out]))


@pytest.mark.parametrize("group", [0, 32, 128])
def test_checkpoint_of_zeros_infinities_and_nan(group):
    x = torch.zeros(4, 300, device=DEV)
    x[1, 5], x[2, 6], x[3, 7] = math.inf, math.nan, 1e-45
    x[1, 6] = x[2, 5] = x[3, 290] = 1.0
    say("checkpoint of special values", group)
    c = fff.checkpoint(x, group)
    r = fff.restore(c, torch.float32)
    g = group or 300
    assert bool((r[0] == 0).all()) and bool((c.scale[0] == O.TINY).all())
    assert math.isinf(float(c.scale[1, 0])) and bool(r[1, :min(g, 300)].isnan().all())
    assert math.isnan(float(c.scale[2, 0])) and bool(r[2, :min(g, 300)].isnan().all())
    if group:
        assert bool((r[1:3, g:] == 0).all())
    assert float(r[3, 290]) == 1.0 or abs(float(r[3, 290]) - 1) < 1e-6


def test_norm_output_is_a_checkpoint():
    gen = seeded("norm")
    x, w = randn(gen, 40, 200, ty="bf16"), randn(gen, 200, ty="bf16")
    say("norm's output as a checkpoint")
    n = fff.rms_norm(x, w, out_dtype=O.F8, group=64)
    c = fff.Checkpoint(n.y, n.scale, 64)
    assert torch.equal(fff.restore(c, torch.float32).to(F64), O.load(n.y, n.scale, 64))
    dy, W = randn(gen, 40, 96, ty="bf16"), randn(gen, 200, 96, ty="bf16")
    o = fff.linear_backward(dy, c, W, want_dx=False)
    again = fff.linear_backward(dy, fff.restore(c), W, want_dx=False)
    assert torch.equal(o.dW, again.dW) and o.dx is None


# ---- how it is called ----

@pytest.mark.parametrize("ty,out", TYPES)
@pytest.mark.parametrize("T,K,N", [(1, 256, 512), (40, 300, 70), (300, 64, 256)])
def test_y_in_the_residuals_place(T, K, N, ty, out):
    gen = seeded(T, K, N)
    say("linear in place", T, K, N, ty, out)
    x, W, r = randn(gen, T, K, ty=ty), randn(gen, K, N, ty=ty), randn(gen, T, N, ty=out)
    want = fff.linear(x, W, residual=r).y
    got = fff.linear(x, W, residual=r, y=r).y
    assert got is r and torch.equal(got, want)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(1, 128, 256), (33, 72, 136), (300, 64, 256), (257, 41, 77)])
def test_views_anywhere_and_nothing_beside_them(T, K, N, ty):
    """Tensors that start one element into a buffer: the same values, and what
    lies before and behind the outputs is left as it was."""
    gen = seeded(T, K, N)
    say("views", T, K, N, ty)

    def odd(t):
        buf = torch.full((t.numel() + 65,), 7.0, device=DEV).to(t.dtype)
        v = buf[1:1 + t.numel()].view(t.shape)
        v.copy_(t)
        return v, buf

    x, W, W2, dy = (odd(randn(gen, *s, ty=ty))[0] for s in ((T, K), (K, N), (K, N), (T, N)))
    outs = {}

    def out(name, *shape, f32=False):
        v, buf = odd(torch.zeros(*shape, dtype=torch.float32 if f32 else TY[ty], device=DEV))
        outs[name] = (v, buf)
        return v

    fff.linear(x, W, y=out("y", T, N), act="silu")
    fff.gated(x, W, W2, h=out("h", T, N))
    fff.linear_backward(dy, x, W, dx=out("dx", T, K), dW=out("dW", K, N, f32=True),
                        dbias=out("dbias", N, f32=True))
    fff.gated_backward(dy, x, W, W2, dy, dy, dx=out("dx2", T, K), dW_gate=out("dWg", K, N, f32=True),
                       dW_up=out("dWu", K, N, f32=True), h=out("h2", T, N))
    torch.cuda.synchronize()
    for name, (v, buf) in outs.items():
        assert float(buf[0]) == 7.0 and bool((buf[1 + v.numel():] == 7.0).all()), name
    x, W, W2, dy = (t.clone() for t in (x, W, W2, dy))
    y, ey = O.linear(d64(x), d64(W), None, None, "silu")[2:]
    O.close(outs["y"][0], y, ey + (y.abs() + ey) * U[ty], "y")
    h, eh = O.gated(d64(x), d64(W), d64(W2), "silu")[4:]
    O.close(outs["h"][0], h, eh + (h.abs() + eh) * U[ty], "h")
    dx, ex = O.product(d64(dy), d64(W).t())
    O.close(outs["dx"][0], dx, ex + (dx.abs() + ex) * U[ty], "dx")


def test_no_rows():
    say("no rows")
    for ty in ("f32", "bf16"):
        x, W = torch.empty(0, 40, dtype=TY[ty], device=DEV), torch.ones(40, 24, dtype=TY[ty], device=DEV)
        dy = torch.empty(0, 24, dtype=TY[ty], device=DEV)
        assert fff.linear(x, W).y.shape == (0, 24) and fff.gated(x, W, W).h.shape == (0, 24)
        o = fff.linear_backward(dy, x, W, want_dbias=True)
        assert o.dx.shape == (0, 40) and bool((o.dW == 0).all()) and bool((o.dbias == 0).all())
        g = fff.gated_backward(dy, x, W, W, dy, dy, want_h=True)
        assert bool((g.dW_gate == 0).all()) and bool((g.dW_up == 0).all()) and g.h.shape == (0, 24)
        c = fff.checkpoint(x)
        assert c.codes.shape == (0, 40) and fff.restore(c).shape == (0, 40)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(5, 100, 200), (200, 72, 264)])
def test_a_bad_row_stays_alone(T, K, N, ty):
    """NaN and infinity in one row of x or dy reach that row of y, h and dx
    only, and one column of a weight that column only."""
    gen = seeded(T, K, N)
    say("a bad row", T, K, N, ty)
    x, W, dy = randn(gen, T, K, ty=ty), randn(gen, K, N, ty=ty), randn(gen, T, N, ty=ty)
    bad = x.clone()
    bad[3, 7], bad[4, 9] = math.nan, math.inf
    rest = [i for i in range(T) if i not in (3, 4)]
    for f in (lambda v: fff.linear(v, W).y, lambda v: fff.gated(v, W, W).h):
        good, got = f(x), f(bad)
        assert torch.equal(good[rest], got[rest]) and bool(got[3].isnan().all())
        assert not bool(got[4].isfinite().any())
    bdy = dy.clone()
    bdy[3, 7] = math.nan
    good, got = fff.linear_backward(dy, x, W).dx, fff.linear_backward(bdy, x, W).dx
    rest = [i for i in range(T) if i != 3]
    assert torch.equal(good[rest], got[rest]) and bool(got[3].isnan().all())
    Wb = W.clone()
    Wb[11, 13] = math.inf
    cols = [i for i in range(N) if i != 13]
    assert torch.equal(fff.linear(x, W).y[:, cols], fff.linear(x, Wb).y[:, cols])


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(1, 512, 256), (40, 1000, 96), (600, 264, 136)])
def test_the_same_on_every_call_and_stream(T, K, N, ty):
    gen = seeded(T, K, N)
    say("streams", T, K, N, ty)
    x, W, dy = randn(gen, T, K, ty=ty), randn(gen, K, N, ty=ty), randn(gen, T, N, ty=ty)

    def everything(stream=None):
        a = fff.linear(x, W, act="gelu", save="e4m3", stream=stream)
        b = fff.gated(x, W, W, save="same", stream=stream)
        c = fff.linear_backward(dy, x, W, act="gelu", pre=a.pre, want_dbias=True, stream=stream)
        d = fff.gated_backward(dy, x, W, W, b.gate, b.up, want_h=True, stream=stream)
        return [a.y, a.pre.codes.float(), a.pre.scale, b.h, b.gate, b.up, *c, *d]

    first = everything()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    # two at once
    both = [everything(s) for s in streams]
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        both.append(everything())
    torch.cuda.synchronize()
    for other in both:
        assert all(torch.equal(a, b) for a, b in zip(first, other))


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(1, 512, 256), (40, 1000, 96), (600, 264, 136)])
def test_captured(T, K, N, ty):
    """A captured forward and backward, replayed with eager work and new
    inputs between, gives what eager calls give."""
    gen = seeded(T, K, N)
    say("captured", T, K, N, ty)
    x, W, dy = randn(gen, T, K, ty=ty), randn(gen, K, N, ty=ty), randn(gen, T, N, ty=ty)

    def everything():
        a = fff.linear(x, W, act="gelu", save="e4m3")
        b = fff.gated(x, W, W, save="same")
        c = fff.linear_backward(dy, x, W, act="gelu", pre=a.pre, want_dbias=True)
        d = fff.gated_backward(dy, x, W, W, b.gate, b.up, want_h=True)
        return [a.y, a.pre.codes, a.pre.scale, b.h, b.gate, b.up, *c, *d]

    everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = everything()
    for k in range(4):
        x.copy_(randn(gen, T, K, ty=ty))
        dy.copy_(randn(gen, T, N, ty=ty))
        graph.replay()
        torch.cuda.synchronize()
        want = everything()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a.float(), b.float()), k


def test_offsets_past_32_bits():
    """Rows whose elements start past 2^31: the last ones against a call on
    them alone."""
    T, K, N = (1 << 31) // 4096 + 300, 32, 4096
    gen = seeded("large")
    say("offsets past 2^31", T, K, N)
    x = torch.randn(T, K, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    W = randn(gen, K, N, ty="bf16")
    y = fff.linear(x, W, act="silu").y
    tail = fff.linear(x[-300:].clone(), W, act="silu").y
    assert torch.equal(y[-300:], tail)
    c = fff.checkpoint(y, 128)
    t = fff.checkpoint(tail, 128)
    assert torch.equal(c.codes[-300:].float(), t.codes.float()) and torch.equal(c.scale[-300:], t.scale)
    r = fff.restore(c)
    assert torch.equal(r[-300:], fff.restore(t))
    del c
    g = fff.gated_backward(y, None, W, W, r, r, want_dW=False, want_h=True)
    gt = fff.gated_backward(tail, None, W, W, r[-300:].clone(), r[-300:].clone(), want_dW=False, want_h=True)
    assert torch.equal(g.h[-300:], gt.h)
    # (a long batch's dx may be summed in other slices than a short one's)
    d = (g.dx[-300:].double() - gt.dx.double()).abs()
    assert bool((d <= 2 * U["bf16"] * gt.dx.double().abs() + 1e-2 * gt.dx.double().square().mean().sqrt()).all())


# ---- gradients against differences ----

@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_gradients_against_differences(act):
    """Central differences of the float64 forward, step 1e-4: its error is of
    the order of 1e-8 of the sums' sizes, the float32 backward's some 1e-6."""
    gen = seeded("differences", act)
    T, K, N = 6, 9, 10
    say("differences", act)
    x, Wg, Wu, dh = (randn(gen, *s) for s in ((T, K), (K, N), (K, N), (T, N)))
    fwd = fff.gated(x, Wg, Wu, act=act, save="same")
    o = fff.gated_backward(dh, x, Wg, Wu, fwd.gate, fwd.up, act=act)
    lin = fff.linear(x, Wg, act=act, save="same")
    p = fff.linear_backward(dh, x, Wg, act=act, pre=lin.pre if act != "none" else None, want_dbias=True)
    args = [t.to(F64) for t in (x, Wg, Wu)]
    bias = torch.zeros(N, dtype=F64, device=DEV)

    def value(kind, x, Wg, Wu, bias):
        g = x @ Wg + bias
        h = O.activation(g, act)[0]
        return float(((h * (x @ Wu) if kind == "gated" else h) * dh.to(F64)).sum())

    def differences(kind, k):
        every = [a.clone() for a in args] + [bias.clone()]
        flat, out = every[k].view(-1), []
        for i in range(flat.numel()):
            at = float(flat[i])
            flat[i] = at + 1e-4
            up = value(kind, *every)
            flat[i] = at - 1e-4
            out.append((up - value(kind, *every)) / 2e-4)
            flat[i] = at
        return torch.tensor(out, dtype=F64, device=DEV).view(every[k].shape)

    for kind, k, got in (("gated", 0, o.dx), ("gated", 1, o.dW_gate), ("gated", 2, o.dW_up),
                         ("linear", 0, p.dx), ("linear", 1, p.dW), ("linear", 3, p.dbias)):
        want = differences(kind, k)
        assert float((got.to(F64) - want).norm() / want.norm()) < 1e-5, (kind, k)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_slopes_of_large_values(act, ty):
    """Far from zero an activation is the value itself or nothing, and its
    slope 1 or 0, up to infinity."""
    say("large values", act, ty)
    at = torch.tensor([1e2, 1e10, 1e19, 1e20, 3e38, math.inf], device=DEV)
    pre = torch.cat([at, -at]).to(TY[ty]).expand(5, 12).contiguous()
    dy, W = torch.full((5, 12), 2.0, dtype=TY[ty], device=DEV), torch.eye(12, dtype=TY[ty], device=DEV)
    da = fff.linear_backward(dy, None, W, act=act, pre=pre, want_dW=False).dx
    assert bool((da[:, :6] == 2.0).all()) and bool((da[:, 6:] == 0.0).all())
    one = torch.ones_like(pre)
    g = fff.gated_backward(dy, None, W, W, pre[:, :5].repeat(1, 3)[:, :12].contiguous(), one, act=act, want_dW=False,
                           want_h=True)
    # (dx is not compared: dup = dh * 3e38 = 6e38 is beyond float32, and infinite beside weights of 0)
    assert torch.equal(g.h[:, :5], pre[:, :5])
    y = fff.linear(pre[:, :5].contiguous(), torch.eye(5, dtype=TY[ty], device=DEV), act=act).y
    assert torch.equal(y, pre[:, :5])
    y = fff.linear(-pre[:, :5].contiguous(), torch.eye(5, dtype=TY[ty], device=DEV), act=act).y
    assert bool((y == 0).all())


def test_two_calls_at_once_and_stale_workspaces():
    """Few rows with K cut: calls on two streams at once, and on workspaces that
    hold whatever another call left there, its own words among it."""
    gen = seeded("at once")
    T, K, N = 3, 4096, 512
    say("two at once")
    x, W, r = randn(gen, T, K, ty="bf16"), randn(gen, K, N, ty="bf16"), randn(gen, T, N, ty="bf16")
    want = fff.linear(x, W, residual=r).y
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.full((8 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    outs = [r.clone() for _ in range(40)]
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        fff.linear(x, W, residual=y, y=y, workspace=spaces[i % 2], stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in outs)
