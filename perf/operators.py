"""The operators around an FFF layer in a training or serving step, as measured
work: the root-mean-square norm with the residual's addition (also with its
output in 8 bits), its backward pass, the AdamW step over many tensors with
states in 32 or in 8 bits, and the gradient's global norm.

``run`` computes them in a plain form (elementary torch operations in 32 bits)
or, with ``own`` set, through this repository's entry points.  ``exact`` is the
same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
F32, F64, BF16, F8 = torch.float32, torch.float64, torch.bfloat16, torch.float8_e4m3fn
TYPES = {"f32": F32, "bf16": BF16}
EPS = 1e-6
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest scale
BLOCK = 128  # elements of one block of an 8-bit state
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 1e-4, 0.9, 0.999, 1e-8, 0.01, 1000
MAX_NORM = 1.0


def listed():
    return [
        # One token of a decode step in front of a layer of width 2048.
        dict(name="norm_token", op="norm", T=1, d=2048, dtype="bf16", stream="bf16", residual=True,
             out="same", group=0, offset=0.0),
        # A training or prefill batch of 8 x 2048 tokens.
        dict(name="norm_prefill", op="norm", T=16384, d=2048, dtype="bf16", stream="bf16",
             residual=True, out="same", group=0, offset=0.0),
        # 64 requests decoding, the norm's output in 8 bits with a scale for each token.
        dict(name="norm_8bit_decode", op="norm", T=64, d=2048, dtype="bf16", stream="bf16",
             residual=True, out="e4m3", group=0, offset=0.0),
        # A prefill batch with the residual stream in 32 bits, a scale for every 128 columns, the
        # last group and the batch ragged.
        dict(name="norm_8bit_ragged", op="norm", T=16381, d=2040, dtype="bf16", stream="f32",
             residual=True, out="e4m3", group=128, offset=1.0),
        # The backward pass of the training batch, the residual's gradient joined.
        dict(name="norm_back_train", op="norm_back", T=16384, d=2048, dtype="bf16", stream="bf16",
             residual=True, offset=0.0),
        # An odd width and an odd batch near the 768-wide layer's, in 32 bits.
        dict(name="norm_back_ragged", op="norm_back", T=8191, d=767, dtype="f32", stream="f32",
             residual=False, offset=0.0),
        # The smallest layer (64 wide, 2 trees of depth 3): five small tensors.
        dict(name="adamw_tiny", op="adamw", d=64, P=2, D=3, h=32, layers=1, param="f32",
             grad="f32", master=False, state="f32", stochastic=False),
        # A layer of the 2048-wide model, bf16 weights with 32-bit masters.
        dict(name="adamw_layer_2048", op="adamw", d=2048, P=32, D=6, h=128, layers=1, param="bf16",
             grad="f32", master=True, state="f32", stochastic=False),
        # The same layer, both moments in 8 bits.
        dict(name="adamw_8bit_layer_2048", op="adamw", d=2048, P=32, D=6, h=128, layers=1,
             param="bf16", grad="f32", master=True, state="8bit", stochastic=True),
        # Twelve layers of the 768-wide model: 60 tensors from 768 to 0.8 M elements, bf16 weights
        # without masters, everything rounded stochastically.
        dict(name="adamw_8bit_12_layers", op="adamw", d=768, P=16, D=5, h=64, layers=12,
             param="bf16", grad="f32", master=False, state="8bit", stochastic=True),
        # The clipping norm of the smallest layer and of the 2048-wide one.
        dict(name="grad_norm_tiny", op="grad_norm", d=64, P=2, D=3, h=32, layers=1, grad="f32"),
        dict(name="grad_norm_layer_2048", op="grad_norm", d=2048, P=32, D=6, h=128, layers=1,
             grad="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["norm", "norm", "norm_back", "adamw", "adamw", "grad_norm"])
        if op in ("norm", "norm_back"):
            dtype = rng.choice(["bf16", "f32"])
            c = dict(op=op, T=_log(rng, 1, 32768), d=_log(rng, 64, 8192), dtype=dtype,
                     stream=rng.choice(["f32", dtype]), residual=rng.random() < 0.75,
                     offset=rng.choice([0.0, 1.0]))
            if op == "norm":
                c["out"] = rng.choice(["same", "e4m3"])
                c["group"] = rng.choice([0, 32, 64, 128]) if c["out"] == "e4m3" else 0
        else:
            c = dict(op=op, d=_log(rng, 64, 2048), P=rng.randint(1, 32), D=rng.randint(1, 7),
                     h=_log(rng, 16, 128), layers=_log(rng, 1, 12), grad=rng.choice(["f32", "f32", "bf16"]))
            if op == "adamw":
                c["param"] = rng.choice(["f32", "bf16"])
                c["master"] = c["param"] == "bf16" and rng.random() < 0.5
                c["state"] = rng.choice(["f32", "8bit"])
                c["stochastic"] = c["state"] == "8bit" and rng.random() < 0.7
        if work(c)["bytes"] <= most:
            return c


def _sizes(c):
    """Element counts of the trained tensors: node rows, biases, node outputs, the projection
    and the norm's gain of each layer."""
    N = 2 ** (c["D"] + 1) - 1
    return [c["P"] * N * c["d"], c["P"] * N, c["P"] * N * c["h"], c["P"] * c["h"] * c["d"],
            c["d"]] * c["layers"]


def work(c):
    if c["op"] in ("norm", "norm_back"):
        n, e, s = c["T"] * c["d"], 2 if c["dtype"] == "bf16" else 4, 4 if c["stream"] == "f32" else 2
        if c["op"] == "norm":
            # x (the stream's own type without a residual), r, z, y, w; the scales and rstd
            b = n * ((e + 2 * s) if c["residual"] else s) + c["d"] * e + 4 * c["T"]
            b += n * (1 if c["out"] == "e4m3" else e)
            if c["out"] == "e4m3":
                b += 4 * c["T"] * (-(-c["d"] // c["group"]) if c["group"] else 1)
            return {"bytes": b, "flops": 6 * n}
        # dy, z, (dres), w, rstd; dz, (dx where the types differ), dw
        b = n * (e + 2 * s + (s if c["residual"] else 0) + (e if e != s else 0))
        return {"bytes": b + c["d"] * (e + 4) + 4 * c["T"], "flops": 10 * n}
    n = sum(_sizes(c))
    g = 2 if c["grad"] == "bf16" else 4
    if c["op"] == "grad_norm":
        return {"bytes": n * g + 8, "flops": 2 * n}
    p = 8 if c["param"] == "f32" else 10 if c["master"] else 4
    if c["state"] == "f32":
        b = n * (p + g + 16)
    else:
        b = n * (p + g + 4) + 16 * sum(-(-k // BLOCK) for k in _sizes(c))
    return {"bytes": b, "flops": 15 * n}


# ---- inputs ----

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=F32)


def _nearest(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(F8)


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"c": c}
    if c["op"] in ("norm", "norm_back"):
        T, d, ty, st = c["T"], c["d"], TYPES[c["dtype"]], TYPES[c["stream"]]
        s["w"] = (1.0 - c["offset"] + 0.1 * _randn(gen, d)).to(ty)
        # A stream whose columns have scales of their own and whose rows differ in size.
        col = torch.exp(0.5 * _randn(gen, d))
        row = torch.exp(0.5 * _randn(gen, T, 1))
        s["r"] = (_randn(gen, T, d) * col * row).to(st)
        if c["op"] == "norm":
            s["x"] = (0.3 * _randn(gen, T, d)).to(ty) if c["residual"] else None
            s["y"] = torch.empty(T, d, dtype=F8 if c["out"] == "e4m3" else ty, device=DEV)
            s["z"] = torch.empty(T, d, dtype=st, device=DEV) if c["residual"] else None
        else:
            s["rstd"] = torch.rsqrt(s["r"].float().square().mean(1) + EPS)
            s["dy"] = (1e-3 * _randn(gen, T, d)).to(ty)
            s["dres"] = (1e-3 * _randn(gen, T, d)).to(st) if c["residual"] else None
        return s
    # One buffer of each kind for all tensors, each tensor starting on a whole block.
    sizes = _sizes(c)
    first, total = [], 0
    for n in sizes:
        first.append(total)
        total += -(-n // BLOCK) * BLOCK
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)
    for a, n in zip(first, sizes):
        inside[a:a + n] = True

    def cut(buf, k=1):
        return [buf[a // k:a // k + -(-n // k)] for a, n in zip(first, sizes)]

    s["grads"] = (1e-3 * _randn(gen, total) * inside).to(TYPES[c["grad"]])
    s["g"] = cut(s["grads"])
    if c["op"] == "adamw":
        w = 0.02 * _randn(gen, total) * inside
        m = 3e-4 * _randn(gen, total) * inside
        r = 1e-3 * torch.exp(0.3 * _randn(gen, total)) * inside
        flat = {"p": w.to(TYPES[c["param"]]), "master": w if c["master"] else None, "scale": None}
        if c["state"] == "f32":
            flat["m"], flat["v"] = m, r.square()
        else:
            m, r = m.view(-1, BLOCK), r.view(-1, BLOCK)
            sc = torch.stack([m.abs().amax(1), r.amax(1)], 1) / E4M3_MAX
            flat["m"] = _nearest(m / sc[:, :1]).view(-1)
            flat["v"] = _nearest(r / sc[:, 1:]).view(-1)
            flat["scale"] = sc
        s["flat"] = {k: v for k, v in flat.items() if v is not None}
        none = [None] * len(sizes)
        for k in ("p", "m", "v"):
            s[k] = cut(flat[k])
        s["master"] = cut(w) if c["master"] else none
        s["scale"] = cut(flat["scale"], BLOCK) if c["state"] == "8bit" else none
        s["first"], s["sizes"] = first, sizes
        s["factor"] = 0.5 + torch.rand(1, generator=gen, device=DEV)
        s["seed"] = seed * 1000003 + 17 if c["stochastic"] else None
        if c["stochastic"]:  # every element's counter: its place in its tensor, under the tensor's key
            s["counter"] = torch.zeros(total, dtype=torch.int64, device=DEV)
            for t, (a, n) in enumerate(zip(first, sizes)):
                s["counter"][a:a + n] = torch.arange(n, device=DEV) ^ _key(s["seed"], t)
    if own:  # the handle that a program keeps for its tensors
        import sparse_tree_structured_amd as fff
        if c["op"] == "adamw":
            s["table"] = fff.adamw_table(
                s["p"], s["g"], s["m"], s["v"], masters=s["master"] if c["master"] else None,
                scales=s["scale"] if c["state"] == "8bit" else None, weight_decay=DECAY)
        else:
            s["table"] = fff.grad_table(s["g"])
    return s


# ---- one pass ----

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_tree_structured_amd as fff
    c = s["c"]
    if c["op"] == "norm":
        o = fff.rms_norm(s["x"] if c["residual"] else s["r"], s["w"],
                         residual=s["r"] if c["residual"] else None, eps=EPS,
                         weight_offset=c["offset"], group=c["group"], y=s["y"], residual_out=s["z"],
                         want_rstd=True)
        return {"y": o.y, "z": o.residual_out, "scale": o.scale, "rstd": o.rstd}
    if c["op"] == "norm_back":
        o = fff.rms_norm_backward(s["dy"], s["r"], s["w"], s["rstd"], dresidual=s["dres"],
                                  weight_offset=c["offset"])
        return {"dz": o.dz, "dx": o.dx if c["dtype"] != c["stream"] else None, "dw": o.dweight}
    if c["op"] == "grad_norm":
        return fff.grad_norm(s["table"], max_norm=MAX_NORM)
    fff.adamw_step(s["table"], lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, step=STEP,
                   grad_scale=s["factor"], seed=s["seed"])
    return s["flat"]


def _run_plain(s):
    c = s["c"]
    if c["op"] == "norm":
        return _norm_plain(c, s)
    if c["op"] == "norm_back":
        return _norm_back_plain(c, s)
    if c["op"] == "grad_norm":
        norm = s["grads"].float().square().sum().sqrt()
        factor = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
        return torch.stack([norm, torch.where(torch.isfinite(norm), factor, math.nan)])
    _adamw_plain(c, s)
    return s["flat"]


def _grouped(y, group):
    """Rows as whole groups of columns, the last one filled up with zeros."""
    T, d = y.shape
    return torch.nn.functional.pad(y, (0, -d % group)).view(T, -1, group)


def _norm_plain(c, s):
    z = s["r"].float()
    if c["residual"]:
        z = s["x"].float() + z
    rstd = 1.0 / torch.sqrt((z * z).mean(1) + EPS)
    y = z * rstd[:, None] * (s["w"].float() + c["offset"])
    out = {"z": z.to(s["r"].dtype) if c["residual"] else None, "rstd": rstd, "scale": None}
    if c["out"] == "same":
        return {**out, "y": y.to(s["w"].dtype)}
    g = _grouped(y, c["group"] or c["d"])
    scale = (g.abs().amax(2) / E4M3_MAX).clamp(min=TINY)
    q = _nearest(g * (1.0 / scale)[:, :, None]).view(c["T"], -1)[:, :c["d"]]
    return {**out, "y": q.contiguous(), "scale": scale}


def _norm_back_plain(c, s):
    zhat = s["r"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * (s["w"].float() + c["offset"])
    dz = s["rstd"][:, None] * (g - zhat * (g * zhat).mean(1, keepdim=True))
    if c["residual"]:
        dz = dz + s["dres"].float()
    return {"dz": dz.to(s["r"].dtype), "dw": (dy * zhat).sum(0),
            "dx": dz.to(s["dy"].dtype) if c["dtype"] != c["stream"] else None}


def _mix(h):
    """MurmurHash3's 32-bit finaliser on integers below 2^32 (a tensor's or Python's)."""
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _key(seed, t):
    lo, hi = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    return _mix(_mix(lo ^ ((0x9E3779B9 * (t + 1)) & 0xFFFFFFFF)) ^ hi)


def _to_e4m3(x, u):
    """x (at most 448 in size) to e4m3: to nearest, or down or up by the uniforms u."""
    if u is None:
        return x.clamp(-E4M3_MAX, E4M3_MAX)
    a = x.abs()
    e = ((a.view(torch.int32) >> 23) - 127).clamp(min=-6)
    up = ((3 - e + 127) << 23).view(F32)  # 2^(3-e), exact
    down = ((e - 3 + 127) << 23).view(F32)
    return torch.copysign((torch.floor(a * up + u) * down).clamp(max=E4M3_MAX), x)


def _to_blocks(x, u):
    """A moment over its blocks' scales, its e4m3 values, and the scales."""
    b = x.view(-1, BLOCK)
    scale = (b.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
    t = (b * (1.0 / scale)[:, None]).view(-1)
    return t, _to_e4m3(t, u).to(F8), scale


def _adamw_plain(c, s):
    f = s["flat"]
    step = LR / (1.0 - BETA1 ** STEP)
    root = 1.0 / math.sqrt(1.0 - BETA2 ** STEP)
    g = s["grads"].float() * s["factor"]
    m, v = f["m"].float(), f["v"].float()
    if c["state"] == "8bit":
        m = (m.view(-1, BLOCK) * f["scale"][:, :1]).view(-1)
        v = (v.view(-1, BLOCK) * f["scale"][:, 1:]).view(-1).square()
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    r = torch.sqrt(v)
    w = f["master" if c["master"] else "p"].float()
    w = w * (1.0 - LR * DECAY) - step * (m / (r * root + ADAM_EPS))
    if c["master"]:
        f["master"].copy_(w)
    h = _mix(s["counter"]) if c["stochastic"] else None
    if c["stochastic"] and c["param"] == "bf16" and not c["master"]:
        low = (_mix(h ^ 0x9E3779B9) & 0xFFFF).to(torch.int32)
        w = ((w.view(torch.int32) + low) & -65536).view(F32)
    f["p"].copy_(w)
    if c["state"] == "f32":
        f["m"].copy_(m)
        f["v"].copy_(v)
        return
    _, q, f["scale"][:, 0] = _to_blocks(m, None if h is None else (h & 0xFFFF).float() / 65536.0)
    f["m"].copy_(q)
    t, q, f["scale"][:, 1] = _to_blocks(r, None if h is None else (h >> 16).float() / 65536.0)
    # a second moment above zero stays above zero
    f["v"].copy_(torch.where((t > 0) & (q.float() == 0), 2.0 ** -9, q.float()).to(F8))


# ---- the same in 64 bits, from the definitions ----

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        z = s["r"].to(F64) + (s["x"].to(F64) if c["residual"] else 0.0)
        rstd = (z.pow(2).sum(1) / c["d"] + EPS).pow(-0.5)
        y = z * torch.outer(rstd, torch.ones(c["d"], dtype=F64, device=DEV)) * (s["w"].to(F64) + c["offset"])
        out = {"y": y, "z": z if c["residual"] else None, "rstd": rstd, "scale": None}
        if c["out"] == "e4m3":
            # What the 8-bit values stand for: y over its group's scale, before any rounding.
            group = c["group"] or c["d"]
            parts = y.split(group, dim=1)
            out["scale"] = torch.stack([k.abs().max(1).values for k in parts], 1) / E4M3_MAX
            out["y"] = torch.cat([k / out["scale"][:, i:i + 1] for i, k in enumerate(parts)], 1)
        return out
    if c["op"] == "norm_back":
        z, dy, rstd = s["r"].to(F64), s["dy"].to(F64), s["rstd"].to(F64).view(-1, 1)
        g = dy * (s["w"].to(F64) + c["offset"])
        dot = (g * z).sum(1, keepdim=True)
        dz = rstd * g - rstd.pow(3) * z * dot / c["d"]
        if c["residual"]:
            dz = dz + s["dres"].to(F64)
        return {"dz": dz, "dx": dz if c["dtype"] != c["stream"] else None,
                "dw": torch.mv((dy * z).t(), rstd.view(-1))}
    if c["op"] == "grad_norm":
        norm = math.sqrt(sum(float(torch.dot(g.to(F64), g.to(F64))) for g in s["g"]))
        return torch.tensor([norm, min(1.0, MAX_NORM / (norm + 1e-6))], dtype=F64)
    out = {k: torch.zeros(v.shape, dtype=F64, device=DEV) for k, v in s["flat"].items()}
    for t, (a, n) in enumerate(zip(s["first"], s["sizes"])):
        g = s["g"][t].to(F64) * s["factor"].to(F64)
        m, v = s["m"][t].to(F64), s["v"][t].to(F64)
        at = torch.arange(n, device=DEV) // BLOCK
        if c["state"] == "8bit":
            sc = s["scale"][t].to(F64)
            m, v = m * sc[at, 0], (v * sc[at, 1]).pow(2)
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g.pow(2)
        mhat, vhat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        p = (s["master"][t] if c["master"] else s["p"][t]).to(F64)
        p = p - LR * DECAY * p - LR * mhat / (vhat.sqrt() + ADAM_EPS)
        out["p"][a:a + n] = p
        if c["master"]:
            out["master"][a:a + n] = p
        if c["state"] == "8bit":
            # What the codes stand for: the moments over their blocks' scales, before any rounding.
            top = torch.zeros(-(-n // BLOCK), 2, dtype=F64, device=DEV)
            for k, x in enumerate((m.abs(), v.sqrt())):
                top[:, k] = top[:, k].scatter_reduce(0, at, x, "amax")
            top /= E4M3_MAX
            out["scale"][a // BLOCK:a // BLOCK + len(top)] = top
            m, v = m / top[at, 0], v.sqrt() / top[at, 1]
        out["m"][a:a + n] = m
        out["v"][a:a + n] = v
    return out
