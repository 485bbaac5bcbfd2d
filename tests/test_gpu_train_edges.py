"""The norm and the optimiser at the ends of their arguments' ranges, on the
GPU: AdamW bit for bit with its formulas evaluated operation by operation in
32 bits."""
import numpy as np
import pytest
import torch

import sparse_tree_structured_amd as fff
import train_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KW = dict(lr=1.0, beta1=0.9, beta2=0.99)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def same(got, want, what):
    got = got.cpu().numpy()
    eq = (got == want) | (np.isnan(got) & np.isnan(want))
    assert eq.all(), f"{what}: {(~eq).sum()} of {eq.size} differ"


def step_of(p, g, m, v, **kw):
    """A step on the GPU and the same by the formulas: (tensors, oracle)."""
    with np.errstate(all="ignore"):
        o = O.adamw(p, g, m, v, wd=0.0, step=3, **kw)
    t = [dev(a) for a in (p, g, m, v)]
    fff.adamw_step(fff.adamw_table([t[0]], [t[1]], [t[2]], [t[3]]), step=3, **kw)
    return t, o


@pytest.mark.parametrize("eps", [2.0 ** -60, 2.0 ** 59, 2.0 ** 60, 2.0 ** 90, 1e30, 2.0 ** 126, 3e38, 1e39])
def test_an_eps_of_any_size(eps):
    """Weights of zero show the quotient's own bits.  The last eps is infinite
    in 32 bits: the quotient is zero."""
    print(f"[gpu] adamw eps={eps}", flush=True)
    rng = np.random.default_rng(21)
    n = 4096
    size = 2.0 ** rng.uniform(-60, 59, n)
    g = (rng.normal(size=n) * np.minimum(size, 2.0 ** 28)).astype(np.float32)
    m = (rng.normal(size=n) * size).astype(np.float32)
    t, o = step_of(np.zeros(n, np.float32), g, m, rng.random(n).astype(np.float32), eps=eps, **KW)
    same(t[0], o["p"], "param")
    same(t[2], o["m"], "exp_avg")
    same(t[3], o["v"], "exp_avg_sq")
    assert np.isfinite(o["p"]).all()


@pytest.mark.parametrize("bad", [-(2.0 ** -126), -1e-20, -1.0, -1e30, float("nan"), float("-inf")])
def test_a_second_moment_below_zero_is_not_hidden(bad):
    """No step makes one; a damaged state's element becomes NaN, as the root
    of a negative number is, and the others stay as they are."""
    print(f"[gpu] adamw exp_avg_sq={bad}", flush=True)
    rng = np.random.default_rng(22)
    n = 600
    p, m = (rng.normal(size=n).astype(np.float32) for _ in range(2))
    v = rng.random(n).astype(np.float32)
    v[::7] = bad
    t, o = step_of(p, np.zeros(n, np.float32), m, v, eps=1e-8, **KW)
    assert np.isnan(o["p"][::7]).all() and np.isfinite(np.delete(o["p"], np.s_[::7])).all()
    same(t[0], o["p"], "param")
    same(t[2], o["m"], "exp_avg")
    same(t[3], o["v"], "exp_avg_sq")


@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("d", [1, 8, 30, 96, 104, 256, 264, 512, 1000, 1001, 2040])
def test_an_infinite_rstd_gives_infinite_scales_at_every_width(d, group, ty):
    """With eps 0, squares too small for 32 bits leave rstd infinite, and with
    it every output and every scale, whatever lanes the row's end leaves
    idle.  A row of zeros is 0 times infinity: NaN."""
    x = torch.full((3, d), 1e-30, dtype=ty, device=DEV)
    x[1] = 0.0
    x[2] = 1.0
    print(f"[gpu] rms_norm rstd=inf d={d} group={group} {ty}", flush=True)
    o = fff.rms_norm(x, out_dtype=torch.float8_e4m3fn, group=group, eps=0.0, want_rstd=True)
    assert torch.isinf(o.rstd[:2]).all() and o.rstd[2] == 1.0
    assert torch.isinf(o.scale[0]).all() and torch.isnan(o.scale[1]).all()
    assert torch.isnan(o.y[:2].float()).all()
    assert (o.scale[2] == np.float32(1) / np.float32(448)).all() and (o.y[2].float() == 448).all()
