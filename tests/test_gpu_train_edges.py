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


# One launch for rows and columns; two; rows and columns in one again past 16384 columns.  Even and odd widths.
OVER = [(40, 770), (3, 2048), (900, 333), (5000, 770), (3000, 2049), (60, 16400), (50, 16387)]


@pytest.mark.parametrize("T,d", OVER)
def test_backward_of_a_32_bit_stream_over_its_inputs(T, d):
    """dx in the place of dy, and dz in that of z or of the residual's
    gradient, one and all of them at once: the same bits, dweight (which other
    workgroups sum from dy and z) too."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T + d)
    z, dres = (torch.randn(T, d, generator=gen, device=DEV) for _ in range(2))
    dy, w = (torch.randn(*s, generator=gen, device=DEV).bfloat16() for s in ((T, d), (d,)))
    rstd = fff.rms_norm(z, w, want_rstd=True).rstd
    print(f"[gpu] rms_norm_backward over its inputs T={T} d={d}", flush=True)
    want = fff.rms_norm_backward(dy, z, w, rstd, dresidual=dres)
    assert want.dx.dtype == torch.bfloat16 and want.dz.dtype == torch.float32
    assert torch.equal(want.dx, want.dz.bfloat16())
    for over_dy, over in ((True, None), (False, "z"), (True, "z"), (True, "dres"), (False, "dres")):
        t = dict(dy=dy.clone(), z=z.clone(), dres=dres.clone())
        g = fff.rms_norm_backward(t["dy"], t["z"], w, rstd, dresidual=t["dres"], dx=t["dy"] if over_dy else None,
                                  dz=t[over] if over else None)
        assert not over_dy or g.dx.data_ptr() == t["dy"].data_ptr()
        assert not over or g.dz.data_ptr() == t[over].data_ptr()
        assert torch.equal(g.dx, want.dx) and torch.equal(g.dz, want.dz) and torch.equal(g.dweight, want.dweight)


@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(40, 770), (5000, 770), (60, 16400)])
def test_backward_with_dx_and_dz_of_one_type(T, d, ty):
    """Both asked for where the types agree: equal, over the inputs too."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T * d)
    dy, z = (torch.randn(T, d, generator=gen, device=DEV).to(ty) for _ in range(2))
    rstd = fff.rms_norm(z, want_rstd=True).rstd
    print(f"[gpu] rms_norm_backward dx beside dz T={T} d={d} {ty}", flush=True)
    want = fff.rms_norm_backward(dy, z, None, rstd)
    for swap in (False, True):
        a, b = dy.clone(), z.clone()
        g = fff.rms_norm_backward(a, b, None, rstd, dx=b if swap else a, dz=a if swap else b)
        assert torch.equal(a, want.dz) and torch.equal(b, want.dz) and torch.equal(g.dweight, want.dweight)


@pytest.mark.parametrize("T,d", [(5000, 770), (3000, 2049), (40, 770)])
def test_backward_with_a_given_workspace(T, d):
    """Its size as the query says, dirty, and nothing behind it touched."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T - d)
    dy, z = (torch.randn(T, d, generator=gen, device=DEV) for _ in range(2))
    w = torch.randn(d, generator=gen, device=DEV)
    rstd = fff.rms_norm(z, w, want_rstd=True).rstd
    need = fff.rms_norm_backward_workspace_size(T, d, fff.DTYPE_F32, fff.DTYPE_F32)
    assert (need > 0) == (T > 1024)
    want = fff.rms_norm_backward(dy, z, w, rstd)
    print(f"[gpu] rms_norm_backward workspace T={T} d={d}", flush=True)
    buf = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    g = fff.rms_norm_backward(dy, z, w, rstd, workspace=buf[:need])
    assert torch.equal(g.dz, want.dz) and torch.equal(g.dweight, want.dweight)
    assert bool((buf[need:] == 0xFF).all())
    if need:
        with pytest.raises(fff.FFFError) as e:
            fff.rms_norm_backward(dy, z, w, rstd, workspace=buf[:need - 1])
        assert e.value.status == fff.ERROR_WORKSPACE


@pytest.mark.parametrize("before", [False, True])
def test_a_captured_norm_outlives_its_table(before):
    """A table used before the capture or not, then dropped: replays give the
    eager result and touch no tensor that was made since."""
    g = torch.randn(300_000, device=DEV)
    table = fff.grad_table([g])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if before:
        fff.grad_norm(table, stream=side)
        side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = fff.grad_norm(table)
    del table
    with torch.cuda.stream(side):
        other = [torch.full((64,), 7.0, device=DEV) for _ in range(100)]
    other += [torch.full((64,), 7.0, device=DEV) for _ in range(100)]
    print(f"[gpu] grad_norm captured, table dropped, before={before}", flush=True)
    for _ in range(4):
        g.normal_()
        torch.cuda.synchronize()
        want = fff.grad_norm([g])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(bool((o == 7.0).all()) for o in other)


def quotients(m, v, eps):
    """The step's m / (sqrt(v) + eps): betas of one half so late that their
    corrections are 1, weights of zero, no gradient."""
    n = len(m)
    t = [torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), dev(2 * m), dev(2 * v)]
    fff.adamw_step(fff.adamw_table([t[0]], [t[1]], [t[2]], [t[3]]), lr=1.0, step=1000, beta1=0.5, beta2=0.5, eps=eps)
    return -t[0].cpu().numpy()


@pytest.mark.parametrize("first", range(-90, 60, 30))
def test_every_root_of_the_short_form(first):
    """All floats from 2^-90 to 2^60.  A root that is off by its last bit
    shows in the quotient, whose own last bit is finer than the root's for one
    of the two sizes of m."""
    for low in range(first, first + 30, 2):
        print(f"[gpu] adamw root of [2^{low}, 2^{low + 2})", flush=True)
        v = np.arange((127 + low) << 23, (129 + low) << 23, dtype=np.uint32).view(np.float32)
        d = np.sqrt(v) + np.float32(2.0 ** -60)
        for m in (np.float32(1.0), np.float32(1.9999999)):
            assert np.array_equal(quotients(np.full(len(v), m), v, 2.0 ** -60), m / d)


@pytest.mark.parametrize("size", [-60, 0, 59])
def test_the_quotient_of_every_mantissa(size):
    """Every mantissa of m over the smallest and the largest mantissas of a
    divisor and some between (v = 0: the divisor is eps)."""
    rng = np.random.default_rng(23)
    m = np.arange(127 << 23, 128 << 23, dtype=np.uint32).view(np.float32)
    zero = np.zeros_like(m)
    ends = [k for i in range(4) for k in (i, (1 << 23) - 1 - i)]
    print(f"[gpu] adamw quotient over 2^{size}", flush=True)
    for k in ends + list(rng.integers(0, 1 << 23, 8)):
        d = np.float32((1 + int(k) * 2.0 ** -23) * 2.0 ** size)
        assert np.array_equal(quotients(m, zero, float(d)), m / d), k
