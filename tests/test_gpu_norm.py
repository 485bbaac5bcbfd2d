"""The root-mean-square norm and its backward pass on the GPU against the
float64 formulas.

Tolerances.  A row's sum of squares is added in chains of at most 32 products
per lane (four chunks of eight), six steps over a wavefront and sixteen
wavefronts: under 64 roundings, each of which can move the sum by 2^-24 of
itself, and rstd by half of that; z, rstd, and the products of y add fewer
than ten more.  So |y - y64| <= 64 * 2^-24 |y64| in 32 bits, plus one rounding
to the output's type (2^-8 relative for bf16)."""
import numpy as np
import pytest
import torch

import sparse_tree_structured_amd as fff
import train_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TY = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
SLACK = 64 * O.U32


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def randn(rng, shape, ty, size=1.0):
    return torch.from_numpy((rng.normal(size=shape) * size).astype(np.float32)).to(TY[ty]).to(DEV)


def inputs(T, d, ty, st, residual=True, seed=0):
    rng = np.random.default_rng(seed + 7 * T + d)
    x = randn(rng, (T, d), ty if residual else st)
    r = randn(rng, (T, d), st, 2.0) if residual else None
    w = randn(rng, (d,), ty)
    return x, r, w


def close(got, want, bound, what):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {(err - bound)[bad].max()}"


def check_forward(o, x, r, w, eps, offset, ty, st):
    z, rstd, y = O.rms_norm(f64(x), f64(r), f64(w), eps, offset)
    if r is not None:
        close(f64(o.residual_out), z, np.abs(z) * (O.U32 + O.u_of(st)), "residual_out")
    if o.rstd is not None:
        close(f64(o.rstd), rstd, rstd * SLACK, "rstd")
    if o.y.dtype != F8:
        close(f64(o.y), y, np.abs(y) * (SLACK + O.u_of(ty) * 1.01), "y")
    return z, rstd, y


def check_e4m3(o, y, group):
    """Scales within the slack; every code is the nearest one of a value
    within the slack of y / scale."""
    T, d = y.shape
    want = np.maximum(O.group_amax(y, group) / 448, O.TINY)
    scale = f64(o.scale)
    assert scale.shape == want.shape
    close(scale, want, want * SLACK + 2.0 ** -149, "scale")
    t = y / np.repeat(scale, group or d, axis=1)[:, :d]
    code = o.y.view(torch.uint8).cpu().numpy()
    got = O.E4M3[code]
    lo = O.E4M3[O.e4m3_nearest(t * (1 - 2 * SLACK))]
    hi = O.E4M3[O.e4m3_nearest(t * (1 + 2 * SLACK))]
    assert ((got == lo) | (got == hi)).all()


PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("ty,st", PAIRS)
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (1, 64), (5, 65), (2, 511), (9, 512), (4, 513),
                                 (7, 767), (3, 1025), (1, 2048), (70, 2048), (3, 2049), (2, 4099),
                                 (2, 8192), (2, 8193), (1, 16385), (2, 32768)])
def test_forward(T, d, ty, st):
    x, r, w = inputs(T, d, ty, st)
    print(f"[gpu] rms_norm T={T} d={d} {ty} {st}", flush=True)
    o = fff.rms_norm(x, w, residual=r, eps=1e-6, want_rstd=True)
    torch.cuda.synchronize()
    check_forward(o, x, r, w, 1e-6, 0.0, ty, st)


@pytest.mark.parametrize("ty,st", PAIRS)
@pytest.mark.parametrize("T,d", [(1, 40), (300, 768), (2, 5000)])
def test_forward_without_residual_and_weight_offset(T, d, ty, st):
    x, _, w = inputs(T, d, ty, st, residual=False)
    print(f"[gpu] rms_norm alone T={T} d={d} {ty} {st}", flush=True)
    o = fff.rms_norm(x, w, weight_offset=1.0, eps=1e-3)
    assert o.residual_out is None and o.rstd is None and o.scale is None
    check_forward(o, x, None, w, 1e-3, 1.0, ty, st)
    o = fff.rms_norm(x)  # no weight: the layer's type is x's
    assert o.y.dtype == x.dtype
    check_forward(o, x, None, None, 1e-6, 0.0, st, st)


@pytest.mark.parametrize("ty,st", PAIRS)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 30), (5, 129), (64, 768), (2, 2047), (33, 2048),
                                 (2, 4100), (1, 9001)])
def test_forward_e4m3(T, d, group, ty, st):
    x, r, w = inputs(T, d, ty, st, seed=1)
    print(f"[gpu] rms_norm e4m3 T={T} d={d} group={group} {ty} {st}", flush=True)
    o = fff.rms_norm(x, w, residual=r, out_dtype=F8, group=group, want_rstd=True)
    _, _, y = check_forward(o, x, r, w, 1e-6, 0.0, ty, st)
    check_e4m3(o, y, group)


@pytest.mark.parametrize("group", [0, 32])
def test_e4m3_zero_rows_tiny_rows_and_non_finite(group):
    """A zero row has scale 2^-126 and zeros; a row whose outputs are far
    below the smallest scale stays finite; NaN and infinity stay in their
    groups' scales."""
    d = 96
    x = torch.ones(5, d, device=DEV)
    w = torch.ones(d, device=DEV)
    x[0] = 0.0
    x[1] = 1e-3
    x[2, 40] = float("nan")
    x[3, 40] = float("inf")
    w[:32] = 1e-39  # below 448 * 2^-126 over a group of its own
    o = fff.rms_norm(x, w, out_dtype=F8, group=group, eps=1e-6)
    s, y = f64(o.scale), f64(o.y)
    assert (s[0] == O.TINY).all() and (y[0] == 0).all()
    assert np.isfinite(s[[0, 1, 4]]).all() and np.isfinite(y[[0, 1, 4]]).all()
    if group:
        assert s[4, 0] == O.TINY and (np.abs(y[4, :32]) <= 448).all()
    # the row's mean is NaN: so is every output and every scale
    assert np.isnan(s[2]).all() and np.isnan(y[2]).all()
    # an infinite row has rstd 0: zeros, and NaN where infinity meets it
    assert np.isnan(y[3, 40]) and np.isnan(s[3, 40 // group if group else 0])
    plain = f64(fff.rms_norm(x, torch.ones(d, device=DEV)).y)
    assert np.isnan(plain[2]).all() and np.isnan(plain[3, 40]) and (np.delete(plain[3], 40) == 0).all()


def test_in_place_and_views():
    """The residual updated in place, y over x, and tensors that start at odd
    elements of their buffers."""
    T, d = 37, 1001
    for ty in ("bf16", "f32"):
        x, r, w = inputs(T, d, ty, ty, seed=2)
        want = fff.rms_norm(x, w, residual=r)
        buf = torch.zeros(3 * T * d + 16, dtype=TY[ty], device=DEV)
        a, b = buf[1:1 + T * d].view(T, d), buf[3 + T * d:3 + 2 * T * d].view(T, d)
        wv = torch.zeros(d + 1, dtype=TY[ty], device=DEV)[1:]
        a.copy_(x), b.copy_(r), wv.copy_(w)
        o = fff.rms_norm(a, wv, residual=b, residual_out=b, y=a)
        assert o.y.data_ptr() == a.data_ptr() and o.residual_out.data_ptr() == b.data_ptr()
        assert torch.equal(a, want.y) and torch.equal(b, want.residual_out)
        assert buf[0] == 0 and (buf[1 + T * d:3 + T * d] == 0).all() and (buf[3 + 2 * T * d:] == 0).all()


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("d", [5, 257, 513, 769, 1025, 1030, 2051, 4097])
def test_in_place_at_ragged_ends(d, ty):
    """Widths whose last columns start another wavefront's or chunk's access,
    so that two of them hold some columns: in place gives the same bits."""
    T = 2000
    x, r, w = inputs(T, d, ty, ty, seed=4)
    want = fff.rms_norm(x, w, residual=r, want_rstd=True)
    dres = randn(np.random.default_rng(d), (T, d), ty)
    grad = fff.rms_norm_backward(x, want.residual_out, w, want.rstd, dresidual=dres)
    print(f"[gpu] in place d={d} {ty}", flush=True)
    for _ in range(3):
        a, b, c = x.clone(), r.clone(), dres.clone()
        o = fff.rms_norm(a, w, residual=b, residual_out=b, y=a, want_rstd=True)
        assert torch.equal(a, want.y) and torch.equal(b, want.residual_out) and torch.equal(o.rstd, want.rstd)
        g = fff.rms_norm_backward(x, b, w, o.rstd, dresidual=c, dz=c)
        assert torch.equal(c, grad.dz) and torch.equal(g.dweight, grad.dweight)


@pytest.mark.parametrize("ty,st", PAIRS)
@pytest.mark.parametrize("T,d", [(1, 1), (1, 2048), (3, 70), (50, 512), (17, 513), (1030, 100),
                                 (700, 767), (1500, 2048), (40, 3001), (5, 8192), (3, 8200),
                                 (2, 32768), (22000, 100), (5000, 511), (6000, 513), (5001, 767),
                                 (1500, 3001), (600, 8192), (300, 8200), (300, 16400), (70, 32768),
                                 (1000, 2500), (1024, 2048), (1025, 2048), (1000, 1000), (400, 16384),
                                 (400, 12289), (300, 16385), (200, 20001)])
def test_backward(T, d, ty, st):
    """dz within 64 roundings of its terms' sizes (the dot's chains are the
    sum of squares' above); dw is added over at most ceil(T / 1024) rows (a
    quarter of it at narrow widths) and then over 256 partials at most."""
    rng = np.random.default_rng(T + d)
    z, w = randn(rng, (T, d), st), randn(rng, (d,), ty)
    dy, dres = randn(rng, (T, d), ty, 0.1), randn(rng, (T, d), st, 0.1)
    rstd = torch.from_numpy(O.rms_norm(None, f64(z), None, 1e-6, 0.0)[1].astype(np.float32)).to(DEV)
    print(f"[gpu] rms_norm_backward T={T} d={d} {ty} {st}", flush=True)
    for res, offset in ((dres, 0.0), (None, 1.0)):
        o = fff.rms_norm_backward(dy, z, w, rstd, dresidual=res, weight_offset=offset)
        dz, dw, size, wsum = O.rms_norm_backward(f64(dy), f64(z), f64(w), f64(rstd), f64(res), offset)
        close(f64(o.dz), dz, size * SLACK + np.abs(dz) * O.u_of(st) * 1.01, "dz")
        close(f64(o.dx), dz, size * SLACK + np.abs(dz) * O.u_of(ty) * 1.01, "dx")
        close(f64(o.dweight), dw, wsum * (64 + T / 1024 + 256) * O.U32, "dweight")
        assert (o.dx is o.dz) == (ty == st)


@pytest.mark.parametrize("ty,st", PAIRS)
@pytest.mark.parametrize("T,d", [(3, 767), (1100, 5), (1100, 767), (1100, 2047), (1100, 2048),
                                 (1100, 4099)])
def test_backward_of_an_infinite_weight(T, d, ty, st):
    """An infinite weight in the last column makes every row's mean infinite:
    dz is infinite elsewhere, against the signs of z and of the mean, in both
    kernels and in every lane, and dw stays finite."""
    x, _, w = inputs(T, d, ty, st, residual=False)
    z = torch.where(x == 0, torch.ones_like(x), x)  # no zero times infinity
    dy = torch.ones(T, d, dtype=TY[ty], device=DEV)
    w[-1] = float("inf")
    rstd = torch.rsqrt((z.float() ** 2).mean(1) + 1e-6)
    print(f"[gpu] rms_norm_backward of an infinite weight T={T} d={d} {ty} {st}", flush=True)
    g = fff.rms_norm_backward(dy, z, w, rstd)
    got, s = f64(g.dz)[:, :-1], np.sign(f64(z))
    want = -s[:, :-1] * s[:, -1:] * np.inf
    assert (got == want).all()
    assert torch.isfinite(g.dweight).all()


def test_backward_against_differences_of_the_forward():
    """d/dh of sum(y dy) + sum(z dres) along random directions, from the
    library's own float32 forward: central differences with h = 2^-6 have a
    truncation error of about h^2 of the third derivative (here under 1e-3 of
    the terms' sizes) and rounding of 2^-24 sqrt(n) / h."""
    T, d = 6, 200
    rng = np.random.default_rng(5)
    z, w, dy, dres = (randn(rng, s, "f32") for s in ((T, d), (d,), (T, d), (T, d)))
    o = fff.rms_norm(z, w, want_rstd=True)
    g = fff.rms_norm_backward(dy, z, w, o.rstd, dresidual=dres)

    def f(z, w):
        return float((f64(fff.rms_norm(z, w).y) * f64(dy)).sum() + (f64(z) * f64(dres)).sum())

    h = 2.0 ** -6
    for k in range(4):
        ez, ew = randn(rng, (T, d), "f32"), randn(rng, (d,), "f32")
        size = np.abs(f64(g.dz) * f64(ez)).sum()
        assert abs((f(z + h * ez, w) - f(z - h * ez, w)) / (2 * h) - (f64(g.dz) * f64(ez)).sum()) < 2e-3 * size
        size = np.abs(f64(g.dweight) * f64(ew)).sum()
        assert abs((f(z, w + h * ew) - f(z, w - h * ew)) / (2 * h) - (f64(g.dweight) * f64(ew)).sum()) < 1e-4 * size


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", [(40, 770), (3, 2048), (5000, 770)])
def test_backward_over_its_inputs(T, d, ty):
    """dz in the place of dy, z or the residual's gradient, small and large:
    the same bits, dweight (which reads dy and z) too."""
    rng = np.random.default_rng(T)
    z, w, dy, dres = (randn(rng, s, ty) for s in ((T, d), (d,), (T, d), (T, d)))
    rstd = fff.rms_norm(z, w, want_rstd=True).rstd
    want = fff.rms_norm_backward(dy, z, w, rstd, dresidual=dres)
    for k in range(3):
        t = [dy.clone(), z.clone(), dres.clone()]
        g = fff.rms_norm_backward(t[0], t[1], w, rstd, dresidual=t[2], dz=t[k])
        assert torch.equal(t[k], want.dz) and torch.equal(g.dweight, want.dweight)


def test_backward_in_place_without_dweight_and_same_every_time():
    T, d = 6000, 770
    rng = np.random.default_rng(6)
    z, w, dy, dres = (randn(rng, s, "bf16") for s in ((T, d), (d,), (T, d), (T, d)))
    rstd = fff.rms_norm(z, w, want_rstd=True).rstd
    first = fff.rms_norm_backward(dy, z, w, rstd, dresidual=dres)
    for _ in range(3):
        again = fff.rms_norm_backward(dy, z, w, rstd, dresidual=dres)
        assert torch.equal(first.dz, again.dz) and torch.equal(first.dweight, again.dweight)
    alone = fff.rms_norm_backward(dy, z, w, rstd, dresidual=dres, want_dweight=False)
    assert alone.dweight is None and torch.equal(first.dz, alone.dz)
    into = dres.clone()
    fff.rms_norm_backward(dy, z, w, rstd, dresidual=into, dz=into)
    assert torch.equal(first.dz, into)


@pytest.mark.parametrize("mb", [100, 260])
@pytest.mark.parametrize("ty,st,d", [("bf16", "bf16", 4099), ("bf16", "bf16", 4096), ("bf16", "f32", 2051),
                                     ("f32", "f32", 2048)])
@pytest.mark.parametrize("out", [None, F8])
def test_forward_of_large_batches_past_the_caches(mb, ty, st, d, out):
    """A batch large enough for streaming writes, and reads, against its rows
    a part at a time (which are not)."""
    T = (mb << 20) // (d * ((4 if ty == "f32" else 2) * (1 if out else 2) + 2 * (4 if st == "f32" else 2)))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(d)
    x = torch.randn(T, d, generator=gen, device=DEV).to(TY[ty])
    r = torch.randn(T, d, generator=gen, device=DEV).to(TY[st])
    w = torch.randn(d, generator=gen, device=DEV).to(TY[ty])
    kw = dict(out_dtype=out, group=64 if out else 0, want_rstd=True)
    print(f"[gpu] rms_norm large T={T} d={d} {ty} {st} {out}", flush=True)
    o = fff.rms_norm(x, w, residual=r, **kw)
    n = T // 8 + 1
    for a in range(0, T, n):
        part = fff.rms_norm(x[a:a + n], w, residual=r[a:a + n], **kw)
        assert torch.equal(o.y[a:a + n].view(torch.uint8), part.y.view(torch.uint8))
        assert torch.equal(o.residual_out[a:a + n], part.residual_out) and torch.equal(o.rstd[a:a + n], part.rstd)
        assert out is None or torch.equal(o.scale[a:a + n], part.scale)


@pytest.mark.parametrize("ty,st,d", [("bf16", "bf16", 4099), ("bf16", "bf16", 4096), ("f32", "f32", 2051),
                                     ("bf16", "f32", 2050), ("bf16", "f32", 2048)])
def test_backward_of_large_batches_past_the_caches(ty, st, d):
    """A batch large enough for streaming reads against its rows a part at a
    time (which are not), and dweight against the parts' sum."""
    T = (180 << 20) // (d * 3 * (2 if ty == "bf16" else 4))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(d)
    dy, z, dres = (torch.randn(T, d, generator=gen, device=DEV).to(TY[k]) for k in (ty, st, st))
    w = torch.randn(d, generator=gen, device=DEV).to(TY[ty])
    rstd = fff.rms_norm(z, w, want_rstd=True).rstd
    print(f"[gpu] rms_norm_backward large T={T} d={d} {ty}", flush=True)
    g = fff.rms_norm_backward(dy, z, w, rstd, dresidual=dres)
    dw, n = torch.zeros(d, dtype=torch.float64, device=DEV), T // 4 + 1
    for a in range(0, T, n):
        part = fff.rms_norm_backward(dy[a:a + n], z[a:a + n], w, rstd[a:a + n], dresidual=dres[a:a + n])
        assert torch.equal(g.dz[a:a + n], part.dz) and torch.equal(g.dx[a:a + n], part.dx)
        dw += part.dweight.double()
    size = (dy.float().abs() * z.float().abs() * rstd[:, None]).sum(0).double()
    assert bool(((g.dweight.double() - dw).abs() <= size * 2 * (64 + T / 512 + 256) * O.U32).all())


def test_no_rows():
    w = torch.ones(64, device=DEV)
    x = torch.empty(0, 64, device=DEV)
    o = fff.rms_norm(x, w, residual=x, want_rstd=True)
    assert o.y.shape == (0, 64) and o.rstd.shape == (0,)
    assert fff.rms_norm(x, w, out_dtype=F8, group=32).scale.shape == (0, 2)
    g = fff.rms_norm_backward(x, x, w, torch.empty(0, device=DEV),
                              dweight=torch.full((64,), 7.0, device=DEV))
    assert (g.dweight == 0).all()


def test_rows_past_32_bits_of_elements():
    """More than 2^32 elements: the last rows lie past 32-bit offsets and past
    the largest grid."""
    T, d = (1 << 20) + 70, 4104
    assert T * d > 1 << 32
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    x[-3:] = randn(np.random.default_rng(8), (3, d), "bf16")
    w = randn(np.random.default_rng(9), (d,), "bf16")
    print("[gpu] rms_norm past 2^32 elements", flush=True)
    o = fff.rms_norm(x, w, want_rstd=True)
    small = fff.rms_norm(x[-3:].clone(), w, want_rstd=True)
    assert torch.equal(o.y[-3:], small.y) and torch.equal(o.rstd[-3:], small.rstd)
    assert (o.y[:3] == 0).all() and (o.y[-6:-3] == 0).all()
    del o
    dy = torch.ones_like(x)
    rstd = torch.ones(T, device=DEV)
    g = fff.rms_norm_backward(dy, x, w, rstd, dz=dy)
    small = fff.rms_norm_backward(torch.ones_like(x[-3:]), x[-3:].clone(), w, rstd[-3:].clone())
    assert torch.equal(g.dz[-3:], small.dz)
    close(f64(g.dweight), f64(x[-3:]).sum(axis=0), np.abs(f64(x[-3:])).sum(axis=0) * 400 * O.U32, "dweight")


def test_backward_of_more_wide_rows_than_workgroups():
    """Rows of more than 16384 columns, more of them than one launch has
    workgroups for rows: the last rows and the columns' sums."""
    T, d = (1 << 20) + 3, 16400
    z = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    z[-3:] = randn(np.random.default_rng(1), (3, d), "bf16")
    w = randn(np.random.default_rng(2), (d,), "bf16")
    dy, rstd = torch.ones_like(z), torch.ones(T, device=DEV)
    print("[gpu] rms_norm_backward wide and long", flush=True)
    g = fff.rms_norm_backward(dy, z, w, rstd, dz=dy)
    small = fff.rms_norm_backward(torch.ones_like(z[-3:]), z[-3:].clone(), w, rstd[-3:].clone())
    assert torch.equal(g.dz[-3:], small.dz) and torch.equal(g.dz[0], w) and torch.equal(g.dz[(1 << 20) - 1], w)
    assert torch.equal(g.dweight, small.dweight)  # every other row adds zeros


def test_on_another_stream_and_in_a_graph():
    T, d = 130, 2048
    x, r, w = inputs(T, d, "bf16", "bf16", seed=3)
    dy = torch.ones_like(x)
    want = fff.rms_norm(x, w, residual=r, want_rstd=True)
    grad = fff.rms_norm_backward(dy, want.residual_out, w, want.rstd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = fff.rms_norm(x, w, residual=r, want_rstd=True, stream=side)
    g = fff.rms_norm_backward(dy, o.residual_out, w, o.rstd, stream=side)
    side.synchronize()
    assert torch.equal(o.y, want.y) and torch.equal(g.dz, grad.dz) and torch.equal(g.dweight, grad.dweight)
    xin = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = fff.rms_norm(xin, w, residual=r, want_rstd=True)
        g = fff.rms_norm_backward(dy, o.residual_out, w, o.rstd)
    for k in range(1, 4):
        xin.copy_(x * k)
        want = fff.rms_norm(xin, w, residual=r, want_rstd=True)
        grad = fff.rms_norm_backward(dy, want.residual_out, w, want.rstd)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.y, want.y) and torch.equal(g.dz, grad.dz)
        assert torch.equal(g.dweight, grad.dweight)
