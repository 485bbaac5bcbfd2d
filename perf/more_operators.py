"""The dense feed-forward block beside the FFF layer, as measured work: a matrix
product with bias, activation and residual, the gated pair of projections with
their activation and product, the backward passes of both, and activation
checkpoints in 8 bits, which the forward passes write and the backward passes
read.

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
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest scale


def listed():
    return [
        # The down projection of one token of a decode step onto a 32-bit residual stream.
        dict(name="linear_token", op="linear", T=1, K=8192, N=2048, dtype="bf16", out="f32",
             act="none", bias=False, residual=True, save="none", group=0),
        # The same of a training or prefill batch of 8 x 2048 tokens, the stream in bf16.
        dict(name="linear_prefill", op="linear", T=16384, K=8192, N=2048, dtype="bf16", out="bf16",
             act="none", bias=False, residual=True, save="none", group=0),
        # A first layer with bias and GELU in 32 bits near the 768-wide model's, everything odd, its
        # sums kept in 8 bits for the backward pass.
        dict(name="linear_ragged", op="linear", T=8191, K=767, N=2045, dtype="f32", out="f32",
             act="gelu", bias=True, residual=False, save="e4m3", group=64),
        # The backward pass of the training batch's down projection.
        dict(name="linear_back_train", op="linear_back", T=16384, K=8192, N=2048, dtype="bf16",
             act="none", bias=False, x8=False, group=0, grad="f32"),
        # A small first layer's backward pass (the training example's batch and width) from 8 bits.
        dict(name="linear_back_small", op="linear_back", T=512, K=256, N=1024, dtype="bf16",
             act="gelu", bias=True, x8=True, group=32, grad="bf16"),
        # One token, and 64 requests, of a decode step at the dense block's width (4 x 2048).
        dict(name="gated_token", op="gated", T=1, d=2048, F=8192, dtype="bf16", act="silu",
             save="none", group=0),
        dict(name="gated_decode", op="gated", T=64, d=2048, F=8192, dtype="bf16", act="silu",
             save="none", group=0),
        # A training batch, the gate's and the up projection's sums kept in 8 bits.
        dict(name="gated_train", op="gated", T=16384, d=2048, F=8192, dtype="bf16", act="silu",
             save="e4m3", group=128),
        # Its backward pass from 8 bits, h made again for the down projection's gradient.
        dict(name="gated_back_train", op="gated_back", T=16384, d=2048, F=8192, dtype="bf16",
             act="silu", x8=True, saved="e4m3", group=128, want_h=True, grad="bf16"),
        # An odd block near the 768-wide model's, in 32 bits.
        dict(name="gated_back_ragged", op="gated_back", T=8191, d=767, F=2045, dtype="f32",
             act="gelu", x8=False, saved="same", group=0, want_h=False, grad="f32"),
        # The norm's output of a training batch kept in 8 bits.
        dict(name="checkpoint_train", op="checkpoint", T=16384, d=2048, dtype="bf16", group=128),
        # A ragged batch read back, its last group short.
        dict(name="restore_ragged", op="restore", T=16381, d=2040, dtype="bf16", group=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        op = rng.choice(["linear", "linear", "linear_back", "gated", "gated", "gated_back",
                         "checkpoint", "restore"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        # Half of the widths in whole groups of 8, the others any.
        step = rng.choice([1, 8])
        wide = [step * _log(rng, 64 // step, 8192 // step) for _ in range(2)]
        group = rng.choice([32, 64, 128])
        act = rng.choice(["gelu", "silu", "relu"])
        c = dict(op=op, T=_log(rng, 1, 32768), dtype=dtype)
        if op in ("linear", "linear_back"):
            c.update(K=wide[0], N=wide[1], act=rng.choice(["none", act]), bias=rng.random() < 0.5)
        elif op in ("gated", "gated_back"):
            c.update(d=wide[0], F=wide[1], act=act)
        else:
            c.update(d=wide[0], group=rng.choice([0, group]))
        if op in ("linear", "gated"):
            c["save"] = rng.choice(["none", "same", "e4m3"])
            c["group"] = group if c["save"] == "e4m3" else 0
        if op == "linear":
            c.update(out=rng.choice([dtype, "f32"]), residual=rng.random() < 0.5)
        if op in ("linear_back", "gated_back"):
            c["x8"] = rng.random() < 0.5
            c["grad"] = "f32" if dtype == "f32" else "bf16"
        if op == "linear_back":
            # The sums are there where the activation has a slope: in 8 bits beside an 8-bit x.
            c["group"] = group if c["x8"] else 0
            if c["act"] == "none" and not c["x8"]:
                c["grad"] = "f32"
        if op == "gated_back":
            c.update(saved=rng.choice(["same", "e4m3"]), want_h=rng.random() < 0.5)
            c["group"] = group if c["x8"] or c["saved"] == "e4m3" else 0
        w = work(c)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return c


def _groups(d, group):
    return -(-d // group) if group else 1


def work(c):
    e, T = 2 if c["dtype"] == "bf16" else 4, c["T"]

    def kept(n, how):  # bytes of [T, n] as it is kept for the backward pass
        return {"none": 0, "same": T * n * e,
                "e4m3": T * n + 4 * T * _groups(n, c["group"])}[how]

    if c["op"] in ("checkpoint", "restore"):
        return {"bytes": T * c["d"] * e + kept(c["d"], "e4m3"), "flops": 2 * T * c["d"]}
    if c["op"] == "linear":
        K, N, o = c["K"], c["N"], 4 if c["out"] == "f32" else 2
        b = e * (T * K + K * N + (N if c["bias"] else 0)) + o * T * N * (2 if c["residual"] else 1)
        return {"bytes": b + kept(N, c["save"]), "flops": 2 * T * K * N}
    if c["op"] == "linear_back":
        K, N, g = c["K"], c["N"], 4 if c["grad"] == "f32" else 2
        b = e * (T * N + K * N + T * K) + kept(K, "e4m3" if c["x8"] else "same") + g * K * N
        if c["act"] != "none":
            b += kept(N, "e4m3" if c["x8"] else "same")
        return {"bytes": b + (4 * N if c["bias"] else 0), "flops": 4 * T * K * N}
    d, F = c["d"], c["F"]
    if c["op"] == "gated":
        return {"bytes": e * (T * d + 2 * d * F + T * F) + 2 * kept(F, c["save"]),
                "flops": 4 * T * d * F}
    g = 4 if c["grad"] == "f32" else 2
    b = e * (T * F + 2 * d * F + T * d) + kept(d, "e4m3" if c["x8"] else "same")
    b += 2 * kept(F, c["saved"]) + 2 * g * d * F + (e * T * F if c["want_h"] else 0)
    return {"bytes": b, "flops": 8 * T * d * F}


# ---- inputs ----

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=F32)


def _rows(gen, T, d):
    """Rows as a norm leaves them: columns with gains of their own."""
    return _randn(gen, T, d) * (1.0 + 0.2 * _randn(gen, d))


def _nearest(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(F8)


def _grouped(x, group):
    """Rows as whole groups of columns, the last one filled up with zeros."""
    T, d = x.shape
    return torch.nn.functional.pad(x, (0, -d % group)).view(T, -1, group)


def _save(x, group):
    """x in 8 bits: its codes, and a scale for every group of a row."""
    T, d = x.shape
    g = _grouped(x, group or d)
    scale = (g.abs().amax(2) / E4M3_MAX).clamp(min=TINY)
    codes = _nearest(g * (1.0 / scale)[:, :, None]).view(T, -1)[:, :d]
    return codes.contiguous(), scale


def _load(kept, group):
    """What codes and scales stand for, in 32 bits; a tensor is itself."""
    if torch.is_tensor(kept):
        return kept.float()
    codes, scale = kept
    T, d = codes.shape
    return (_grouped(codes.float(), group or d) * scale[:, :, None]).view(T, -1)[:, :d]


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    ty, T = TYPES[c["dtype"]], c["T"]
    s = {"c": c}

    def weight(k, n):
        return (_randn(gen, k, n) / math.sqrt(k)).to(ty)

    def kept(x, eight):
        return _save(x, c["group"]) if eight else x.to(ty)

    if c["op"] in ("checkpoint", "restore"):
        x = _rows(gen, T, c["d"])
        s["x"] = x.to(ty) if c["op"] == "checkpoint" else _save(x, c["group"])
    elif c["op"] in ("linear", "linear_back"):
        K, N = c["K"], c["N"]
        s["W"] = weight(K, N)
        if c["op"] == "linear":
            s["x"] = _rows(gen, T, K).to(ty)
            s["bias"] = (0.3 * _randn(gen, N)).to(ty) if c["bias"] else None
            s["residual"] = (2.0 * _randn(gen, T, N)).to(TYPES[c["out"]]) if c["residual"] else None
        else:
            s["x"] = kept(_rows(gen, T, K), c["x8"])
            s["dy"] = (1e-3 * _randn(gen, T, N)).to(ty)
            s["pre"] = kept(_rows(gen, T, N), c["x8"]) if c["act"] != "none" else None
    else:
        d, F = c["d"], c["F"]
        s["Wg"], s["Wu"] = weight(d, F), weight(d, F)
        if c["op"] == "gated":
            s["x"] = _rows(gen, T, d).to(ty)
        else:
            s["x"] = kept(_rows(gen, T, d), c["x8"])
            s["gate"] = kept(_rows(gen, T, F), c["saved"] == "e4m3")
            s["up"] = kept(_rows(gen, T, F), c["saved"] == "e4m3")
            s["dh"] = (1e-3 * _randn(gen, T, F)).to(ty)
    return s


# ---- one pass ----

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_tree_structured_amd as fff
    c = s["c"]

    def kept(x):
        return x if x is None or torch.is_tensor(x) else fff.Checkpoint(*x, c["group"])

    def shown(x):
        return (x.codes, x.scale) if isinstance(x, fff.Checkpoint) else x

    if c["op"] == "checkpoint":
        return shown(fff.checkpoint(s["x"], group=c["group"]))
    if c["op"] == "restore":
        return fff.restore(kept(s["x"]), TYPES[c["dtype"]])
    save = dict(save=None if c["save"] == "none" else c["save"],
                group=c["group"]) if "save" in c else {}
    if c["op"] == "linear":
        o = fff.linear(s["x"], s["W"], s["bias"], residual=s["residual"], act=c["act"],
                       out_dtype=TYPES[c["out"]], **save)
        return {"y": o.y, "pre": shown(o.pre)}
    if c["op"] == "linear_back":
        o = fff.linear_backward(s["dy"], kept(s["x"]), s["W"], act=c["act"], pre=kept(s["pre"]),
                                want_dbias=c["bias"], grad_dtype=TYPES[c["grad"]])
        return {"dx": o.dx, "dW": o.dW, "dbias": o.dbias}
    if c["op"] == "gated":
        o = fff.gated(s["x"], s["Wg"], s["Wu"], act=c["act"], **save)
        return {"h": o.h, "gate": shown(o.gate), "up": shown(o.up)}
    o = fff.gated_backward(s["dh"], kept(s["x"]), s["Wg"], s["Wu"], kept(s["gate"]), kept(s["up"]),
                           act=c["act"], want_h=c["want_h"], grad_dtype=TYPES[c["grad"]])
    return {"dx": o.dx, "dWg": o.dW_gate, "dWu": o.dW_up, "h": o.h}


def _act(a, how):
    if how == "none":
        return a
    if how == "relu":
        return a.clamp(min=0.0)
    if how == "silu":
        return a / (1.0 + torch.exp(-a))
    return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)))


def _slope(a, how):
    if how == "none":
        return torch.ones_like(a)
    if how == "relu":
        return (a > 0.0).to(a.dtype)
    if how == "silu":
        q = 1.0 / (1.0 + torch.exp(-a))
        return q * (1.0 + a * (1.0 - q))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (a + 0.044715 * a * a * a))
    return 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * a * a)


def _run_plain(s):
    c = s["c"]
    ty = TYPES[c["dtype"]]

    def kept(a):
        return {"none": None, "same": a.to(ty)}[c["save"]] if c["save"] != "e4m3" else _save(a, c["group"])

    if c["op"] == "checkpoint":
        return _save(s["x"].float(), c["group"])
    if c["op"] == "restore":
        return _load(s["x"], c["group"]).to(ty)
    if c["op"] == "linear":
        a = s["x"].float() @ s["W"].float()
        if c["bias"]:
            a = a + s["bias"].float()
        y = _act(a, c["act"])
        if c["residual"]:
            y = y + s["residual"].float()
        return {"y": y.to(TYPES[c["out"]]), "pre": kept(a)}
    if c["op"] == "gated":
        g, u = s["x"].float() @ s["Wg"].float(), s["x"].float() @ s["Wu"].float()
        return {"h": (_act(g, c["act"]) * u).to(ty), "gate": kept(g), "up": kept(u)}
    x, grad = _load(s["x"], c["group"]), TYPES[c["grad"]]
    if c["op"] == "linear_back":
        da = s["dy"].float()
        if c["act"] != "none":
            da = da * _slope(_load(s["pre"], c["group"]), c["act"])
        return {"dx": (da @ s["W"].float().t()).to(ty), "dW": (x.t() @ da).to(grad),
                "dbias": da.sum(0) if c["bias"] else None}
    g, u, dh = _load(s["gate"], c["group"]), _load(s["up"], c["group"]), s["dh"].float()
    a = _act(g, c["act"])
    dg, du = dh * u * _slope(g, c["act"]), dh * a
    return {"dx": (dg @ s["Wg"].float().t() + du @ s["Wu"].float().t()).to(ty),
            "dWg": (x.t() @ dg).to(grad), "dWu": (x.t() @ du).to(grad),
            "h": (a * u).to(ty) if c["want_h"] else None}


# ---- the same in 64 bits, from the definitions ----

def _exact_act(a, how):
    """The activation and its derivative."""
    if how == "none":
        return a, torch.ones_like(a)
    if how == "relu":
        on = (a > 0).to(F64)
        return a * on, on
    if how == "silu":
        q = torch.sigmoid(a)
        return a * q, q + a * q * (1 - q)
    # GELU in its tanh form: a times the logistic function of 2 z
    k = 2 * math.sqrt(2 / math.pi)
    q = torch.sigmoid(k * (a + 0.044715 * a.pow(3)))
    return a * q, q + a * q * (1 - q) * k * (1 + 0.134145 * a.pow(2))


def _exact_values(x, group):
    if torch.is_tensor(x):
        return x.to(F64)
    codes, scale = x
    at = torch.arange(codes.shape[1], device=DEV) // (group or codes.shape[1])
    return codes.to(F64) * scale.to(F64)[:, at]


def _exact_kept(a, how, group):
    if how == "none":
        return None
    if how == "same":
        return a
    # What the codes stand for: the values over their group's scale, before any rounding.
    parts = a.split(group or a.shape[1], dim=1)
    scale = torch.stack([p.abs().max(1).values for p in parts], 1) / E4M3_MAX
    return torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1), scale


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "checkpoint":
        return _exact_kept(s["x"].to(F64), "e4m3", c["group"])
    x = _exact_values(s["x"], c["group"])
    if c["op"] == "restore":
        return x
    if c["op"] == "linear":
        a = torch.mm(x, s["W"].to(F64))
        if c["bias"]:
            a += s["bias"].to(F64)
        y = _exact_act(a, c["act"])[0]
        if c["residual"]:
            y = y + s["residual"].to(F64)
        return {"y": y, "pre": _exact_kept(a, c["save"], c["group"])}
    if c["op"] == "linear_back":
        da = s["dy"].to(F64)
        if c["act"] != "none":
            da = da * _exact_act(_exact_values(s["pre"], c["group"]), c["act"])[1]
        return {"dx": torch.mm(s["W"].to(F64), da.t()).t().contiguous(),
                "dW": torch.mm(da.t(), x).t().contiguous(),
                "dbias": torch.mv(da.t(), torch.ones(c["T"], dtype=F64, device=DEV)) if c["bias"] else None}
    Wg, Wu = s["Wg"].to(F64), s["Wu"].to(F64)
    if c["op"] == "gated":
        g, u = torch.mm(x, torch.cat([Wg, Wu], 1)).split(c["F"], dim=1)
        return {"h": _exact_act(g, c["act"])[0] * u, "gate": _exact_kept(g, c["save"], c["group"]),
                "up": _exact_kept(u, c["save"], c["group"])}
    a, slope = _exact_act(_exact_values(s["gate"], c["group"]), c["act"])
    u, dh = _exact_values(s["up"], c["group"]), s["dh"].to(F64)
    both = torch.cat([slope * u * dh, a * dh], 1)
    dW = torch.mm(both.t(), x)
    return {"dx": torch.mm(both, torch.cat([Wg, Wu], 1).t()), "dWg": dW[:c["F"]].t().contiguous(),
            "dWu": dW[c["F"]:].t().contiguous(), "h": a * u if c["want_h"] else None}
