"""The AdamW step and the gradient norm on the GPU.  The step is compared bit
for bit with its formulas evaluated in 32 bits operation by operation (the
header promises their order and roundings), 8-bit codes and scales included;
the norm with the float64 sum."""
import math

import numpy as np
import pytest
import torch

import sparse_tree_structured_amd as fff
import train_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KW = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8)
TY = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


def dev(a, ty="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(TY[ty]).to(DEV)


def f32(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def codes(t):
    return t.view(torch.uint8).cpu().numpy().reshape(-1)


def same(got, want, what):
    a, b = np.asarray(got), np.asarray(want)
    eq = (a == b) | (np.isnan(a) & np.isnan(b)) if a.dtype.kind == "f" else a == b
    assert a.shape == b.shape and eq.all(), f"{what}: {(~eq).sum()} of {eq.size} differ"


class Tensors:
    """A list of tensors with their oracle copies."""

    def __init__(self, sizes, param="f32", grad="f32", master=False, bits=32, odd=False, seed=0):
        self.rng = np.random.default_rng(seed)
        self.param, self.grad, self.master, self.bits = param, grad, master, bits
        self.sizes = sizes

        def place(n, ty):  # a view that starts at an odd element of its buffer
            t = torch.zeros(n + 3, dtype=ty, device=DEV)
            return t[1:1 + n] if odd else t[:n]

        self.p, self.g, self.w = [], [], []
        for n in sizes:
            v = dev(self.rng.normal(size=n).astype(np.float32))
            p = place(n, TY[param])
            p.copy_(v)
            w = None
            if master:
                w = place(n, torch.float32)
                w.copy_(v)
            self.p.append(p)
            self.w.append(w)
            self.g.append(place(n, TY[grad]))
        m, v, s = fff.adamw_state(self.p, bits=bits)
        if odd and bits == 8:
            m = [place(n, torch.uint8).view(F8) for n in sizes]
            v = [place(n, torch.uint8).view(F8) for n in sizes]
        elif odd:
            m, v = [place(n, torch.float32) for n in sizes], [place(n, torch.float32) for n in sizes]
        self.m, self.v, self.s = m, v, s
        self.wd = [0.1 if n % 2 else 0.0 for n in sizes]
        self.share = [1.0 if n % 3 else 0.5 for n in sizes]
        self.table = fff.adamw_table(self.p, self.g, m, v, masters=self.w if master else None, scales=s,
                                     weight_decay=self.wd, lr_scale=self.share)
        self.ref = [dict(w=f32(a if b is None else b), m=codes(x) if bits == 8 else f32(x),
                         v=codes(y) if bits == 8 else f32(y),
                         scale=None if s is None else s[i].cpu().numpy())
                    for i, (a, b, x, y) in enumerate(zip(self.p, self.w, m, v))]

    def step(self, step, seed=None, gs=None):
        for g in self.g:
            g.copy_(dev((self.rng.normal(size=g.numel()) *
                         10.0 ** self.rng.uniform(-4, 0, g.numel())).astype(np.float32)))
        scale = None if gs is None else dev(np.array([gs], np.float32))
        print(f"[gpu] adamw {len(self.sizes)} tensors {self.param} {self.grad} master={self.master} "
              f"bits={self.bits} seed={seed}", flush=True)
        fff.adamw_step(self.table, step=step, grad_scale=scale, seed=seed, **KW)
        torch.cuda.synchronize()
        for i, r in enumerate(self.ref):
            kw = dict(KW, lr=KW["lr"] * self.share[i])
            o = O.adamw(r["w"], f32(self.g[i]), r["m"], r["v"], wd=self.wd[i], step=step, gs=gs,
                        scale=r["scale"], seed=seed, tensor=i, param_bf16=self.param == "bf16",
                        master=self.master, **kw)
            at = f"tensor {i} of {len(r['w'])}"
            same(f32(self.p[i]), o["p"], f"param, {at}")
            if self.master:
                same(f32(self.w[i]), o["w"], f"master, {at}")
            if self.bits == 8:
                same(codes(self.m[i]), o["m"], f"exp_avg, {at}")
                same(codes(self.v[i]), o["v"], f"exp_avg_sq, {at}")
                same(self.s[i].cpu().numpy(), o["scale"], f"scale, {at}")
            else:
                same(f32(self.m[i]), o["m"], f"exp_avg, {at}")
                same(f32(self.v[i]), o["v"], f"exp_avg_sq, {at}")
            r.update(w=o["w"] if self.master else o["p"], m=o["m"], v=o["v"], scale=o.get("scale"))


SIZES = [1, 7, 8, 127, 128, 129, 2047, 2048, 2049, 10000]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("seed", [None, 123456789012345])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("param,grad,master", [("f32", "f32", False), ("f32", "bf16", False),
                                               ("bf16", "f32", False), ("bf16", "bf16", False),
                                               ("bf16", "f32", True), ("bf16", "bf16", True)])
def test_steps_bit_for_bit(param, grad, master, odd, seed, bits):
    t = Tensors(SIZES, param, grad, master, bits, odd)
    for step in (1, 2, 3):
        t.step(step, seed=None if seed is None else seed + step, gs=0.37 if step == 2 else None)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_takes(bits):
    sizes = [(37 * i) % 300 + 1 for i in range(120)]
    t = Tensors(sizes, "bf16", "f32", False, bits, seed=3)
    t.step(1, seed=5)


def test_empty_tensors_and_kinds_in_one_list():
    """Tensors of several types in one table, some of them empty."""
    rng = np.random.default_rng(4)
    kinds = [("f32", "f32", False), ("bf16", "f32", True), ("bf16", "bf16", False), ("f32", "bf16", False)]
    lists = {k: [] for k in "pgmvw"}
    ref = []
    for i, n in enumerate([300, 0, 40, 5000, 1, 0, 777, 64]):
        param, grad, master = kinds[i % 4]
        p, g = dev(rng.normal(size=n).astype(np.float32), param), dev(rng.normal(size=n).astype(np.float32), grad)
        w = p.float() if master else None
        for k, v in zip("pgmvw", (p, g, torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), w)):
            lists[k].append(v)
        ref.append(O.adamw(f32(p), f32(g), np.zeros(n, np.float32), np.zeros(n, np.float32), wd=0.01,
                           step=1, tensor=i, param_bf16=param == "bf16", master=master, seed=9, **KW))
    table = fff.adamw_table(lists["p"], lists["g"], lists["m"], lists["v"], masters=lists["w"],
                            weight_decay=0.01)
    fff.adamw_step(table, step=1, seed=9, **KW)
    for i, o in enumerate(ref):
        same(f32(lists["p"][i]), o["p"], f"param {i}")
        same(f32(lists["m"][i]), o["m"], f"exp_avg {i}")
        same(f32(lists["v"][i]), o["v"], f"exp_avg_sq {i}")


@pytest.mark.parametrize("bits", [32, 8])
def test_skipped_when_the_factor_is_nan(bits):
    t = Tensors([200, 3000], "bf16", "f32", True, bits)
    t.step(1, seed=1)
    for g in t.g:
        g[5] = float("nan")
    out = fff.grad_norm(t.table, max_norm=1.0)
    assert torch.isnan(out).all()
    kept = [x.clone() for x in t.p + t.w + t.m + t.v + (t.s or [])]
    fff.adamw_step(t.table, step=2, grad_scale=out[1:], seed=2, **KW)
    for a, b in zip(kept, t.p + t.w + t.m + t.v + (t.s or [])):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    t.step(2, seed=2)


def test_a_moment_keeps_its_mean_and_stays_above_zero():
    """Stochastic rounding is unbiased: over n independent elements the mean
    of the stored moment is within five standard errors (each element is off
    by less than an e4m3 step, an eighth of its size)."""
    n = 128 * 4096
    g = torch.full((n,), 0.77, device=DEV)
    g[::128] = 448 / 13.0  # every block's largest
    g[1::128] = 1e-12      # far below the smallest code
    p = torch.zeros(n, device=DEV)
    m, v, s = fff.adamw_state([p], bits=8)
    fff.adamw_step(fff.adamw_table([p], [g], m, v, scales=s), lr=0.0, step=1, beta1=0.0, beta2=0.0,
                   seed=77)
    at = torch.arange(n, device=DEV) % 128
    for t, k in ((m[0], 0), (v[0], 1)):
        val = (t.float().view(-1, 128) * s[0][:, k:k + 1]).view(-1)[at > 1].double()
        assert len(val.unique()) == 2
        assert abs(float(val.mean()) - 0.77) < 5 * 0.77 / 8 / math.sqrt(len(val))
    assert (v[0].float()[1::128] == 2.0 ** -9).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_nan_stays_with_its_element_and_infinity_is_not_lost(bits):
    """No clipping in front: a NaN gradient makes its own element NaN and
    leaves the rest of its block as it would be; an infinite one is NaN or
    infinite in its element."""
    rng = np.random.default_rng(12)
    w = rng.normal(size=300).astype(np.float32)
    g = rng.normal(size=300).astype(np.float32)
    out = {}
    for bad in (0.0, float("nan"), float("inf")):
        p, gg = dev(w), dev(g)
        gg[70] = bad
        m, v, s = fff.adamw_state([p], bits=bits)
        table = fff.adamw_table([p], [gg], m, v, scales=s)
        for step in (1, 2):
            fff.adamw_step(table, step=step, seed=step, **KW)
        out[str(bad)] = [f32(p), f32(m[0]), f32(v[0])]
    for a, b in zip(out["0.0"], out["nan"]):
        assert np.isnan(b[70]) and np.array_equal(np.delete(a, 70), np.delete(b, 70))
    p, m, v = out["inf"]
    assert not np.isfinite(p[70]) and np.isfinite(p[[0, 127]] if bits == 32 else p[128:]).all()


def test_sizes_beyond_the_short_forms():
    """Moments whose sizes need the long division and root: bit for bit."""
    rng = np.random.default_rng(13)
    n = 4096
    size = 2.0 ** rng.uniform(-140, 120, n)
    size[rng.random(n) < 0.1] = 0.0
    for eps in (1e-8, 0.0, 1e-30):
        kw = dict(KW, eps=eps)
        p, g = rng.normal(size=n).astype(np.float32), (rng.normal(size=n) * size).astype(np.float32)
        m = (g * rng.normal(size=n)).astype(np.float32)
        with np.errstate(over="ignore", under="ignore", invalid="ignore", divide="ignore"):
            v = np.minimum((g * g).astype(np.float32) * rng.random(n).astype(np.float32), 1e38).astype(np.float32)
            o = O.adamw(p, g, m, v, wd=0.0, step=3, **kw)
        t = [dev(a) for a in (p, g, m, v)]
        fff.adamw_step(fff.adamw_table([t[0]], [t[1]], [t[2]], [t[3]]), step=3, **kw)
        same(f32(t[0]), o["p"], f"param, eps {eps}")
        same(f32(t[2]), o["m"], f"exp_avg, eps {eps}")
        same(f32(t[3]), o["v"], f"exp_avg_sq, eps {eps}")


@pytest.mark.parametrize("bits", [32, 8])
def test_large_lists_read_past_the_caches(bits):
    """A list large enough for streaming accesses, its tensors at odd
    elements, against the same tensors a few at a time."""
    sizes = [4_000_001, 3_000_127, 5, 2_500_000]  # 30 or 18 bytes an element
    sizes = sizes + ([] if bits == 32 else [3_000_003])
    state = []
    for n in sizes:
        buf = {"w": torch.empty(n + 1, device=DEV)[1:], "g": torch.empty(n + 3, device=DEV)[3:],
               "p": torch.empty(n + 1, device=DEV, dtype=torch.bfloat16)[1:]}
        buf["w"].normal_()
        buf["g"].normal_()
        buf["p"].copy_(buf["w"])
        buf["m"], buf["v"] = (torch.zeros(n + 1, dtype=torch.float32 if bits == 32 else torch.uint8, device=DEV)[1:]
                              for _ in range(2))
        if bits == 8:
            buf["m"], buf["v"] = buf["m"].view(F8), buf["v"].view(F8)
            buf["s"] = torch.zeros(-(-n // 128), 2, device=DEV)
        state.append(buf)
    other = [{k: v.clone() for k, v in b.items()} for b in state]

    def table(bs):
        return fff.adamw_table([b["p"] for b in bs], [b["g"] for b in bs], [b["m"] for b in bs], [b["v"] for b in bs],
                               masters=[b["w"] for b in bs], scales=[b["s"] for b in bs] if bits == 8 else None)

    for step in (1, 2):
        fff.adamw_step(table(state), step=step, **KW)
        for b in other:
            fff.adamw_step(table([b]), step=step, **KW)
    for a, b in zip(state, other):
        for k in a:
            assert torch.equal(a[k].view(torch.uint8) if a[k].dtype == F8 else a[k],
                               b[k].view(torch.uint8) if b[k].dtype == F8 else b[k]), k
    big = torch.randn(44_000_003, device=DEV)[1:]  # 176 MB
    want = float(big.double().square().sum().sqrt())
    assert abs(float(fff.grad_norm([big])[0]) - want) <= 1.01 * O.U32 * want


def test_elements_past_32_bits():
    """A tensor of more than 2^32 elements: offsets, blocks and random
    numbers of its last elements."""
    n = (1 << 32) + 300
    print("[gpu] adamw past 2^32 elements", flush=True)
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    m = torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8)
    v = torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.zeros(-(-n // 128), 2, device=DEV)
    tail = np.random.default_rng(0).normal(size=300).astype(np.float32)
    p[-300:] = dev(tail, "bf16")
    g[-300:] = dev(tail[::-1].copy(), "bf16")
    a, b = f32(p[-300:]), f32(g[-300:])
    fff.adamw_step(fff.adamw_table([p], [g], [m], [v], scales=[s]), step=1, seed=8, **KW)
    words = O.words
    try:  # the oracle's elements are the tensor's last 300 (2^32 is a multiple of 128)
        O.words = lambda seed, tensor, i: words(seed, tensor, i + (1 << 32))
        zero = np.zeros(300, np.uint8)
        o = O.adamw(a, b, zero, zero, wd=0.0, step=1, scale=np.zeros((3, 2), np.float32), seed=8,
                    param_bf16=True, **KW)
    finally:
        O.words = words
    same(f32(p[-300:]), o["p"], "param")
    same(codes(m[-300:]), o["m"], "exp_avg")
    same(codes(v[-300:]), o["v"], "exp_avg_sq")
    same(s[-3:].cpu().numpy(), o["scale"], "scale")
    assert not bool(p[:1 << 20].any()) and not bool(p[(1 << 32) - (1 << 20):1 << 32].any())
    out = fff.grad_norm([g])
    assert abs(float(out[0]) - np.linalg.norm(b.astype(np.float64))) < 2e-7 * float(out[0])


@pytest.mark.parametrize("sizes", [[1], [5, 16384, 16385, 3], [0, 700], [100003], [50] * 350, [0],
                                   [65536], [65537], [1024] * 64, [1025] * 32, [1] * 65, [60000, 0, 7],
                                   [131072], [131073], [2048] * 64, [2049] * 33])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_grad_norm(sizes, grad):
    """Squares are summed in 64 bits: the result is off by its rounding to 32
    bits alone (2^-24), and the factor by a rounding more."""
    rng = np.random.default_rng(len(sizes))
    g = [dev((rng.normal(size=n + 1) * 10.0 ** rng.uniform(-20, 20)).astype(np.float32), grad)[1:]
         for n in sizes]
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in g))
    print(f"[gpu] grad_norm {len(sizes)} tensors {grad}", flush=True)
    for limit in (0.5 * want if want else 1.0, math.inf):
        out = fff.grad_norm(g, max_norm=limit)
        norm, factor = (float(v) for v in out.cpu())
        assert abs(norm - want) <= 1.01 * O.U32 * want
        assert abs(factor - min(1.0, limit / (want + 1e-6))) <= 2 * O.U32
        assert torch.equal(out, fff.grad_norm(fff.grad_table(g), max_norm=limit))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_grad_norm_not_finite(bad):
    g = [torch.ones(1000, device=DEV), torch.ones(20000, device=DEV)]
    g[1][17777] = bad
    out = fff.grad_norm(g, max_norm=1.0).cpu()
    assert not math.isfinite(float(out[0])) and math.isnan(float(out[1]))
    # squares past the range of 32 bits are still summed; a norm past it is not finite
    big = [torch.full((4,), 1e30, device=DEV)]
    assert abs(float(fff.grad_norm(big)[0]) / 2e30 - 1) < 1e-6
    huge = fff.grad_norm([torch.full((4,), 3e38, device=DEV)]).cpu()
    assert math.isinf(float(huge[0])) and math.isnan(float(huge[1]))


def test_on_another_stream_and_in_a_graph():
    t, u = (Tensors([300, 5000], "bf16", "f32", True, 8, seed=6) for _ in range(2))
    for a, b in zip(t.g, u.g):
        a.normal_()
        b.copy_(a)
    torch.cuda.synchronize()

    def step(x, **kw):
        out = fff.grad_norm(x.table, max_norm=1.0, **kw)
        fff.adamw_step(x.table, step=1, grad_scale=out[1:], seed=4, **KW, **kw)
        return out

    def check():
        torch.cuda.synchronize()
        for a, b in zip(t.p + t.w + t.m + t.v + t.s, u.p + u.w + u.m + u.v + u.s):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))

    side = torch.cuda.Stream()
    kept = step(t), step(u, stream=side)
    check()
    del kept
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(u)
    for _ in range(3):
        step(t)
        graph.replay()
        check()


def test_a_table_keeps_the_workspace_of_a_captured_norm():
    """A norm with a workspace, captured, then used eagerly on two streams:
    every replay gives the eager result and touches nothing else."""
    g = torch.randn(300_000, device=DEV)
    table = fff.grad_table([g])
    side = torch.cuda.Stream()
    fff.grad_norm(table, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = fff.grad_norm(table)
    for k in range(4):
        g.normal_()
        torch.cuda.synchronize()
        want = fff.grad_norm(table)
        other = [torch.full((64,), 7.0, device=DEV) for _ in range(20)]
        fff.grad_norm(table, stream=side)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(bool((o == 7.0).all()) for o in other)
