"""The dense feed-forward operators at sizes that take their large tiles, the
float32 products on bf16 planes among them, against float64 (bounds:
dense_oracle.py)."""
import math

import pytest
import torch

import dense_oracle as O
import sparse_tree_structured_amd as fff
from test_gpu_dense import DEV, check_gated, check_gated_back, check_linear, check_linear_back, randn, say, seeded

pytestmark = pytest.mark.gpu

# Tiles of 256 x 256, 128 x 256 and 128 x 128 with whole and ragged rows,
# columns and ends of K, K in one piece and in slices.
BF16 = [(4096, 512, 4096), (4100, 264, 4104), (8200, 136, 2056), (1000, 2048, 2048), (520, 1032, 1160),
        (2056, 8, 2056), (300, 4104, 520), (16400, 72, 1032)]
# Odd, so through the registers; and float32 beyond and below the split's rule.
ANY = [(3001, 1023, 1537, "f32"), (2048, 1024, 2048, "f32"), (4097, 513, 2045, "bf16"), (700, 300, 900, "f32")]


@pytest.mark.parametrize("T,K,N", BF16)
def test_bf16(T, K, N):
    check_linear(T, K, N, "bf16", "bf16")
    check_linear(T, K, N, "bf16", "bf16", act="gelu", bias=True, residual=True, seed=1)
    check_linear(T, K, N, "bf16", "bf16", act="silu", bias=True, save="e4m3", group=64, seed=2)
    check_linear(T, K, N, "bf16", "f32", act="relu", residual=True, save="same", seed=3)
    for group in (32, 64, 128):
        check_gated(T, K, N, "bf16", save="e4m3", group=group, seed=group)
    check_gated(T, K, N, "bf16", act="gelu", save="same")
    check_gated(T, K, N, "bf16", act="relu")


@pytest.mark.parametrize("T,K,N", BF16)
def test_bf16_backward(T, K, N):
    check_linear_back(T, K, N, "bf16")
    check_linear_back(T, K, N, "bf16", act="gelu", group=64, x_group=128, grad="bf16")
    check_gated_back(T, K, N, "bf16", group=128, x_group=0, grad="bf16")
    check_gated_back(T, K, N, "bf16", act="gelu", want_h=False)


@pytest.mark.parametrize("T,K,N,ty", ANY)
def test_any_type_and_width(T, K, N, ty):
    check_linear(T, K, N, ty, "f32", act="gelu", bias=True, save="e4m3", group=64)
    check_linear(T, K, N, ty, ty, residual=True, seed=1)
    for group in (32, 128):
        check_gated(T, K, N, ty, save="e4m3", group=group, seed=group)
    check_gated(T, K, N, ty, save="same")
    check_linear_back(T, K, N, ty)
    check_linear_back(T, K, N, ty, act="silu", group=32, x_group=0, seed=1)
    check_gated_back(T, K, N, ty)
    check_gated_back(T, K, N, ty, act="gelu", group=64, x_group=64, seed=1)


@pytest.mark.parametrize("one", [False, True])
def test_one_gate_is_kept_without_the_other(one):
    """(through the C entry point: the binding keeps both or neither)"""
    gen = seeded("one gate", one)
    T, K, N = 4096, 256, 2048
    say("gated saving one", one)
    x, Wg, Wu = randn(gen, T, K, ty="bf16"), randn(gen, K, N, ty="bf16"), randn(gen, K, N, ty="bf16")
    both = {s: fff.gated(x, Wg, Wu, save=s, group=32) for s in ("same", "e4m3")}
    h = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    for s, code, group in (("same", fff.DTYPE_BF16, 0), ("e4m3", fff.DTYPE_E4M3, 32)):
        shape = fff.DenseShape(T, K, N, fff.DTYPE_BF16, fff.DTYPE_BF16, fff.ACTS["silu"], code, group, fff.DTYPE_BF16,
                               0, fff.DTYPE_F32)
        want = both[s].up if one else both[s].gate
        codes = torch.zeros_like(want if s == "same" else want.codes)
        scale = torch.zeros_like(want.scale) if s == "e4m3" else None
        kept = [codes.data_ptr(), scale.data_ptr() if scale is not None else 0]
        save = [0, 0, *kept] if one else [*kept, 0, 0]
        h.zero_()
        st = fff.load_library().fff_gated(shape, x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), h.data_ptr(), *save, 0, 0,
                                          stream)
        assert st == fff.SUCCESS
        assert torch.equal(h, both[s].h)
        assert torch.equal(codes.float(), (want if s == "same" else want.codes).float())
        if scale is not None:
            assert torch.equal(scale, want.scale)


@pytest.mark.parametrize("T,K,N", [(3000, 1024, 1600), (4096, 520, 2048)])
def test_bad_values_in_large_float32_products(T, K, N):
    """Where a value is not finite the products are as float32's: infinity
    stays infinity, and nothing else changes beyond rounding.  (On bf16 planes
    infinity times a plane's zero would be NaN.)"""
    gen = seeded("bad", T, K, N)
    say("bad values", T, K, N)
    x, W, r = randn(gen, T, K), randn(gen, K, N), randn(gen, T, N)
    good = fff.linear(x, W, residual=r).y
    bad = x.clone()
    bad[5, 3], bad[T - 1, K - 1], bad[7, 0] = math.inf, -math.inf, math.nan
    y = r.clone()
    fff.linear(bad, W, residual=y, y=y)
    assert bool((y[5] == torch.where(W[3] > 0, math.inf, -math.inf)).all())
    assert bool((y[T - 1] == torch.where(W[K - 1] > 0, -math.inf, math.inf)).all())
    assert bool(y[7].isnan().all())
    rest = [i for i in range(T) if i not in (5, 7, T - 1)]
    bound = O.sum_u(K) * (x.double().abs() @ W.double().abs()) * 2 + good.double().abs() * 2 * O.U32
    O.close(y[rest], good[rest].double(), bound[rest], "the other rows")
    # and again without them: nothing is left over
    assert torch.equal(fff.linear(x, W, residual=r).y, good)
    dy = randn(gen, T, N)
    a = fff.linear_backward(dy, x, W)
    bdy = dy.clone()
    bdy[9, 11] = math.inf
    b = fff.linear_backward(bdy, x, W)
    assert bool((b.dx[9] == torch.where(W[:, 11] > 0, math.inf, -math.inf)).all())
    assert bool((b.dW[:, 11] == torch.where(x[9] > 0, math.inf, -math.inf)).all())
    rest = [i for i in range(T) if i != 9]
    O.close(b.dx[rest], a.dx[rest].double(), 2 * O.sum_u(N) * (dy.double().abs() @ W.double().t().abs())[rest],
            "dx's other rows")
    gate = randn(gen, T, N)
    bg = gate.clone()
    bg[4, 2] = math.nan
    g = fff.gated_backward(dy, x, W, W, bg, gate, want_h=True)
    assert bool(g.dx[4].isnan().all()) and bool(g.dW_gate[:, 2].isnan().all()) and bool(g.h[4, 2].isnan())
    assert bool(g.dx[5].isfinite().all()) and bool(g.dW_gate[:, 3].isfinite().all())


def test_large_float32_values():
    """The planes hold float32's whole range upwards: the largest value, whose
    nearest bf16 is infinite, and sizes down to where the low plane ends."""
    gen = seeded("range")
    T, K, N = 2048, 1024, 2048
    say("range of the planes")
    top = torch.finfo(torch.float32).max
    for size in (top, 1e30, 1e-25):
        x = torch.zeros(T, K, device=DEV)
        x[:, 0] = size
        x[:, 1] = size * 0.7381
        W = torch.zeros(K, N, device=DEV)
        W[:2] = randn(gen, 2, N).clamp(-2, 2) / 8
        y = fff.linear(x, W).y
        want = x[:, :2].double() @ W[:2].double()
        bound = O.sum_u(2) * (x[:, :2].double().abs() @ W[:2].double().abs())
        O.close(y, want, bound, f"size {size}")


def test_captured_and_replayed_float32():
    """The split's word is the captured call's own: values that are not finite
    in one replay and finite ones in the next."""
    gen = seeded("captured planes")
    T, K, N = 2048, 1024, 2048
    say("captured planes")
    x, W = randn(gen, T, K), randn(gen, K, N)
    fff.linear(x, W)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fff.linear(x, W).y
    bound = 2 * O.sum_u(K) * (x.double().abs() @ W.double().abs())
    for k in range(4):
        x[3, 5] = math.inf if k == 1 else 1.0
        graph.replay()
        torch.cuda.synchronize()
        want = fff.linear(x, W).y
        torch.cuda.synchronize()
        assert bool(torch.isinf(y[3]).all()) == (k == 1)
        fine = [i for i in range(T) if i != 3]
        O.close(y[fine], want[fine].double(), bound[fine], f"replay {k}")
