"""The dense feed-forward operators at the edges of what their header allows:
no rows, replays of a captured call, values at the ends of float32's range,
operands anywhere in memory, the workspace's end, calls from several threads,
offsets past 2^31, the widest and the longest sizes (bounds: dense_oracle.py)."""
import concurrent.futures
import math

import pytest
import torch

import dense_oracle as O
import sparse_tree_structured_amd as fff
from test_gpu_dense import (DEV, TY, U, check_gated, check_gated_back, check_linear, check_linear_back, d64, randn, say,
                            seeded)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N", [(4097, 8192), (8191, 8191), (4096, 8192), (65535, 1023), (1023, 65535)])
def test_gradients_of_no_rows_at_wide_weights(K, N):
    say("no rows", K, N)
    for ty in ("bf16", "f32"):
        W = torch.empty(K, N, dtype=TY[ty], device=DEV)
        x, dy = W.new_empty(0, K), W.new_empty(0, N)
        dW, dbias, up = (torch.full(s, 7.0, device=DEV) for s in ((K, N), (N,), (K, N)))
        o = fff.linear_backward(dy, x, W, dW=dW, dbias=dbias)
        assert o.dx.shape == (0, K) and not bool(dW.any()) and not bool(dbias.any())
        g = fff.gated_backward(dy, x, W, W, dy, dy, want_h=True, dW_gate=dW.fill_(7.0), dW_up=up)
        assert g.dx.shape == (0, K) and g.h.shape == (0, N) and not bool(dW.any()) and not bool(up.any())


def test_replays_after_a_value_that_is_not_finite():
    """Large float32 products: a replay gives an eager call's bits, whatever the
    replays before it met."""
    T, K, N = 2048, 1024, 2048
    gen = seeded("replays")
    say("replays after infinity")
    x, W, V, dy = randn(gen, T, K), randn(gen, K, N), randn(gen, K, N), randn(gen, T, N)

    def everything():
        a = fff.linear(x, W, act="silu", save="same")
        b = fff.gated(x, W, V, save="same")
        c = fff.linear_backward(dy, x, W, want_dbias=True)
        d = fff.linear_backward(dy, x, W, act="silu", pre=a.pre)
        e = fff.gated_backward(dy, x, W, V, b.gate, b.up, want_h=True)
        return [a.y, a.pre, b.h, b.gate, b.up, *c, d.dx, d.dW, *e]

    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = everything()
    bad = {1: (x, math.inf), 3: (dy, math.nan), 5: (W, -math.inf)}
    for k in range(7):
        t, value = bad.get(k, (x, 0.5))
        t[3, 5] = value
        graph.replay()
        torch.cuda.synchronize()
        want = everything()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num()), (k, i)
        t[3, 5] = 0.5


def test_finite_values_whose_products_overflow():
    """Large float32 products of one pair of values each: infinity with the
    pair's sign beyond float32's range, and the product below it.  (On bf16
    planes the middle parts' terms have signs of their own.)"""
    T, K, N = 2048, 1024, 2048
    gen = seeded("overflow")
    say("products that overflow")
    most = torch.finfo(torch.float32).max

    def sizes(n, lo, hi):
        v = torch.exp2(lo + (hi - lo) * torch.rand(n, generator=gen, device=DEV, dtype=torch.float64))
        return (v * torch.where(torch.rand(n, generator=gen, device=DEV) < 0.5, -1.0, 1.0)).float()

    def check(got, a, b, what):
        want = a.double()[:, None] * b.double()[None, :]
        over = want.abs() > most
        assert bool(over.any()) and bool((~over).any())
        near = (want.abs() - most).abs() < 2.0 ** -20 * most
        ok = torch.where(over, got.double() == want.sign() * math.inf,
                         (got.double() - want).abs() <= O.sum_u(1) * want.abs() + O.TINY)
        assert bool((ok | near).all()), (what, int((~(ok | near)).sum()))

    def rows(n, k, v):  # [n, k] with v in its first column
        t = torch.zeros(n, k, device=DEV)
        t[:, 0] = v
        return t

    for lo, hi in ((100.0, 127.9), (40.0, 90.0)):
        a, b = sizes(T, lo, hi), sizes(N, 0.0, 89.0)
        check(fff.linear(rows(T, K, a), rows(N, K, b).t().contiguous()).y, a, b, "y")
        g = fff.gated(rows(T, K, a), rows(N, K, b).t().contiguous(), rows(N, K, b).t().contiguous(), act="none",
                      save="same")
        check(g.gate, a, b, "gate")
        check(g.up, a, b, "up")
        c = sizes(K, 0.0, 89.0)
        W = rows(K, N, c)
        check(fff.linear_backward(rows(T, N, a), None, W, want_dW=False).dx, a, c, "dx")
        x, dy = rows(K, T, c).t().contiguous(), rows(N, T, b).t().contiguous()
        dy[0] *= 2.0 ** 30
        check(fff.linear_backward(dy, x, W, want_dx=False).dW, c, dy[0], "dW")


@pytest.mark.parametrize("power", [45.9, 47.1, -108, -115, -122, -129])
def test_the_planes_range(power):
    """Large float32 products of values around the largest that planes take,
    and of small ones: below 2^-110 the low plane ends at 2^-133, bf16's
    smallest step, which moves a value by at most 2^-134."""
    T, K, N = 2048, 1024, 2048
    gen = seeded("planes", power)
    say("range of the planes", power)
    x, W = randn(gen, T, K).clamp(-2, 2), randn(gen, K, N).clamp(-2, 2)
    for a, b in ((power, 0.0 if power > 0 else 40.0), (0.0 if power > 0 else 40.0, power)):
        xs, Ws = (x.double() * 2.0 ** a).float(), (W.double() * 2.0 ** b).float()
        want, bound = O.product(d64(xs), d64(Ws))
        if power < 0:
            bound = bound + 2.0 ** -134 * (d64(xs).abs().sum(1, keepdim=True) + d64(Ws).abs().sum(0, keepdim=True))
        O.close(fff.linear(xs, Ws).y, want, bound + want.abs() * O.U32 + O.TINY, (a, b))


def odd(t):
    """A view with t's values that starts one element into a buffer."""
    buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(33, 72, 136), (257, 41, 77), (300, 64, 256), (1200, 264, 1032), (2048, 1024, 2048)])
def test_every_output_of_operands_at_odd_addresses(T, K, N, ty):
    """All outputs against float64, at widths of whole 16-byte pieces among
    others, whose tiles would go straight into LDS if they were aligned."""
    gen = seeded("odd", T, K, N)
    say("odd addresses", T, K, N, ty)
    x, dy = odd(randn(gen, T, K, ty=ty)), odd(randn(gen, T, N, ty=ty))
    W, V = (odd(randn(gen, K, N, ty=ty, size=1 / math.sqrt(K))) for _ in range(2))
    gate, up = (odd(randn(gen, T, N, ty=ty, size=2.0)) for _ in range(2))
    kept = [fff.checkpoint(t, g) for t, g in ((x, 32), (gate, 64), (up, 64))]
    kept = [fff.Checkpoint(odd(c.codes.view(torch.uint8)).view(c.codes.dtype), odd(c.scale), c.group) for c in kept]

    def out(*shape, f32=False):
        return odd(torch.zeros(*shape, dtype=torch.float32 if f32 else TY[ty], device=DEV))

    u, f = U[ty], O.U32
    y = fff.linear(x, W, act="silu", y=out(T, N)).y
    want, e = O.linear(d64(x), d64(W), None, None, "silu")[2:]
    O.close(y, want, e + (want.abs() + e) * u, "y")
    h = fff.gated(x, W, V, h=out(T, N)).h
    want, e = O.gated(d64(x), d64(W), d64(V), "silu")[4:]
    O.close(h, want, e + (want.abs() + e) * u, "h")
    o = fff.linear_backward(dy, x, W, dx=out(T, K), dW=out(K, N, f32=True), dbias=out(N, f32=True))
    want, e = O.product(d64(dy), d64(W).t())
    O.close(o.dx, want, e + (want.abs() + e) * u, "dx")
    want, e = O.product(d64(x).t(), d64(dy))
    O.close(o.dW, want, e + (want.abs() + e) * f, "dW")
    O.close(o.dbias, d64(dy).sum(0), O.sum_u(T) * d64(dy).abs().sum(0), "dbias")
    for keep in (False, True):
        a, b, c = kept if keep else (x, gate, up)
        xv, g, w = (O.load(t.codes, t.scale, t.group) if keep else d64(t) for t in (a, b, c))
        o = fff.gated_backward(dy, a, W, V, b, c, dx=out(T, K), dW_gate=out(K, N, f32=True),
                               dW_up=out(K, N, f32=True), h=out(T, N))
        value, slope, ev, es = O.activation(g, "silu")
        d = d64(dy)
        dg, du = d * w * slope, d * value
        eg = (d * w).abs() * es + dg.abs() * 3 * f
        eu = d.abs() * ev + du.abs() * 2 * f
        eg, eu = eg + (dg.abs() + eg) * u, eu + (du.abs() + eu) * u
        want, e = O.product(torch.cat([dg, du], 1), torch.cat([d64(W), d64(V)], 1).t(), torch.cat([eg, eu], 1))
        O.close(o.dx, want, e + (want.abs() + e) * u, "the pair's dx")
        ex = xv.t().abs() * u if keep and ty == "bf16" else None
        for got, da, ea, what in ((o.dW_gate, dg, eg, "dW_gate"), (o.dW_up, du, eu, "dW_up")):
            want, e = O.product(xv.t(), da, ex, ea)
            O.close(got, want, e + (want.abs() + e) * f, what)
        e = ev * w.abs() + (value * w).abs() * 2 * f
        O.close(o.h, value * w, e + ((value * w).abs() + e) * u, "h made again")


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(1, 4096, 264), (40, 1000, 96), (70, 96, 200), (257, 41, 77), (520, 1032, 1160),
                                   (1000, 1023, 1537), (2048, 1024, 2048)])
def test_a_workspace_of_the_queried_size(T, K, N, ty):
    """Calls on workspaces of just the bytes asked for, full of NaN: the values
    of calls on their own ones, and nothing behind the end is written.  dW is
    the same with and without dx."""
    gen = seeded("workspace", T, K, N)
    say("workspaces", T, K, N, ty)
    x, dy, W, V = (randn(gen, *s, ty=ty) for s in ((T, K), (T, N), (K, N), (K, N)))
    x8 = fff.checkpoint(x, 64)
    code = {"f32": fff.DTYPE_F32, "bf16": fff.DTYPE_BF16}[ty]
    space = torch.full((1 << 28,), 255, dtype=torch.uint8, device=DEV)

    def shape(save=None, act="none", x_kept=False):
        return (T, K, N, code, code, fff.ACTS[act], fff.DTYPE_E4M3 if save else code, save or 0,
                fff.DTYPE_E4M3 if x_kept else code, 64 if x_kept else 0)

    def run(name, sizes, call):
        need = fff._dense(name, *sizes)[1]
        want = call(None)
        got = call(space[:need])
        torch.cuda.synchronize()
        assert bool((space[need:] == 255).all()), name
        space[:need] = 255
        for a, b in zip(want, got):
            if a is not None:
                assert torch.equal(a.float(), b.float()), name

    def flat(o):
        return [t for part in o for t in ((part.codes, part.scale) if isinstance(part, fff.Checkpoint) else (part,))]

    a = fff.linear(x, W, act="gelu", save="e4m3", group=32)
    b = fff.gated(x, W, V, save="e4m3", group=128)
    run("fff_linear", shape() + (code,), lambda ws: fff.linear(x, W, workspace=ws))
    run("fff_linear", shape(32, "gelu") + (code,),
        lambda ws: flat(fff.linear(x, W, act="gelu", save="e4m3", group=32, workspace=ws)))
    run("fff_gated", shape(128, "silu") + (code,),
        lambda ws: flat(fff.gated(x, W, V, save="e4m3", group=128, workspace=ws)))
    back = dict(want_dbias=True, grad_dtype=TY[ty])
    run("fff_linear_backward", shape() + (code,), lambda ws: fff.linear_backward(dy, x, W, workspace=ws, **back))
    for grads in (dict(), dict(want_dx=False), dict(want_dW=False)):
        run("fff_linear_backward", shape(32, "gelu", True) + (code,),
            lambda ws: fff.linear_backward(dy, x8, W, act="gelu", pre=a.pre, workspace=ws, **back, **grads))
        run("fff_gated_backward", shape(128, "silu", True) + (code,),
            lambda ws: fff.gated_backward(dy, x8, W, V, b.gate, b.up, want_h=True, grad_dtype=TY[ty], workspace=ws,
                                          **grads))
    both = fff.gated_backward(dy, x, W, V, b.gate, b.up)
    assert torch.equal(both.dW_up, fff.gated_backward(dy, x, W, V, b.gate, b.up, want_dx=False).dW_up)
    assert torch.equal(both.dx, fff.gated_backward(dy, None, W, V, b.gate, b.up, want_dW=False).dx)


def test_calls_of_several_host_threads():
    """One stream and one size to a thread, small and large ones, each again and
    again beside the others: the values of calls by themselves."""
    say("host threads")
    sizes = [(3, 4096, 512, "bf16"), (64, 2048, 768, "f32"), (600, 264, 136, "bf16"), (2048, 1024, 2048, "f32")]
    work = []
    for T, K, N, ty in sizes:
        gen = seeded("threads", T, K, N)
        x, W, dy = randn(gen, T, K, ty=ty), randn(gen, K, N, ty=ty), randn(gen, T, N, ty=ty)

        def calls(stream=None, x=x, W=W, dy=dy):
            g = fff.gated(x, W, W, save="same", stream=stream)
            return [fff.linear(x, W, residual=dy, act="silu", stream=stream).y, g.h,
                    *fff.gated_backward(dy, x, W, W, g.gate, g.up, want_h=True, stream=stream)]

        work.append((calls, calls(), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def many(item):
        calls, want, stream = item
        got = [calls(stream) for _ in range(20)]
        stream.synchronize()
        return all(torch.equal(a, b) for g in got for a, b in zip(g, want))

    with concurrent.futures.ThreadPoolExecutor(len(work)) as pool:
        assert all(pool.map(many, work))


def test_offsets_past_32_bits_on_planes():
    """Large float32 products whose operands, planes among them, have elements
    past 2^31: rows at the end against calls on them alone, sums over all rows
    against those over two parts of them."""
    T, K, N = (1 << 20) + 300, 512, 2056
    gen = seeded("planes past 2^31")
    say("planes past 2^31")
    assert T * N > 1 << 31
    dh, gate = (torch.randn(T, N, generator=gen, device=DEV) for _ in range(2))
    x, W, V = randn(gen, T, K), randn(gen, K, N, size=N ** -0.5), randn(gen, K, N, size=N ** -0.5)
    o = fff.gated_backward(dh, x, W, V, gate, gate, act="relu", want_h=True)
    tail = slice(T - 300, T)
    c = [t[tail].clone() for t in (dh, x, gate)]
    p = fff.gated_backward(c[0], c[1], W, V, c[2], c[2], act="relu", want_h=True)
    assert torch.equal(o.h[tail], p.h)
    dg, du = c[0] * c[2] * (c[2] > 0), c[0] * c[2].clamp(min=0)
    size = d64(dg).abs() @ d64(W).abs().t() + d64(du).abs() @ d64(V).abs().t()
    O.close(o.dx[tail], d64(p.dx), 2 * O.sum_u(2 * N) * size, "dx")
    parts, half = [], T // 2
    for rows in (slice(0, half), slice(half, T)):
        q = fff.gated_backward(dh[rows], x[rows], W, V, gate[rows], gate[rows], act="relu", want_dx=False)
        parts.append((d64(q.dW_gate), d64(q.dW_up)))
    for k, got in enumerate((o.dW_gate, o.dW_up)):
        da = dh * gate.clamp(min=0)  # (relu with the gate as up: dg = du)
        size = x.abs().t() @ da.abs_()
        del da
        O.close(got, parts[0][k] + parts[1][k], 2.1 * O.sum_u(T) * d64(size), ("dW_gate", "dW_up")[k])
    del o, p, q, gate, parts, size
    B = W.t().contiguous()
    y = fff.linear(dh, B, residual=x).y
    want, e = O.product(d64(c[0]), d64(B))
    want = want + d64(c[1])
    O.close(y[tail], want, e + want.abs() * 2 * O.U32, "y")
    O.close(y[tail], d64(fff.linear(c[0], B, residual=c[1]).y), 2 * e + want.abs() * 4 * O.U32, "y of the rows alone")
    del dh, y, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N", [(1, 1 << 20, 8), (1, 8, 1 << 20), (70, (1 << 20) - 1, 40), (70, 40, (1 << 20) - 1),
                                   ((1 << 20) + 3, 3, 2)])
def test_the_widest_and_the_longest(T, K, N, ty):
    check_linear(T, K, N, ty, ty, act="silu", bias=True, save="e4m3", group=32)
    check_gated(T, K, N, ty)
    check_linear_back(T, K, N, ty, act="gelu", group=32, x_group=0)
    check_gated_back(T, K, N, ty, group=64, x_group=32)
