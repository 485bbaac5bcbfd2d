"""The dense feed-forward operators at the edges of what their header allows:
no rows, replays of a captured call."""
import math

import pytest
import torch

import sparse_tree_structured_amd as fff
from test_gpu_dense import DEV, TY, randn, say, seeded

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
