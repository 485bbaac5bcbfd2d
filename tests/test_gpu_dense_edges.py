"""The dense feed-forward operators at the edges of what their header allows:
no rows, replays of a captured call, values at the ends of float32's
range (bounds: dense_oracle.py)."""
import math

import pytest
import torch

import dense_oracle as O
import sparse_tree_structured_amd as fff
from test_gpu_dense import DEV, TY, d64, randn, say, seeded

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
