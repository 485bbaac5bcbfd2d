"""Plain numpy forms of the operators around the layer (norm, AdamW, gradient
norm), written from their formulas and apart from the kernels: in 64 bits
where a result is compared within a bound, and operation by operation in 32
bits where the library promises the bits.  CPU only."""
from __future__ import annotations

import math

import numpy as np

U32 = 2.0 ** -24   # relative rounding error of float32
UBF16 = 2.0 ** -8  # of bfloat16
TINY = 2.0 ** -126


def u_of(dtype: str) -> float:
    return {"f32": U32, "bf16": UBF16}[dtype]


# ---- e4m3 (OCP) ----

def e4m3_table() -> np.ndarray:
    """The values of the 256 codes in float64 (0x7f and 0xff are NaN)."""
    v = np.empty(256)
    for c in range(128):
        e, m = c >> 3, c & 7
        v[c] = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    v[127] = np.nan
    v[128:] = -v[:128]
    return v


E4M3 = e4m3_table()
_POS = E4M3[:127]
_MID = (_POS[1:] + _POS[:-1]) / 2


def e4m3_nearest(t: np.ndarray) -> np.ndarray:
    """Codes (uint8) nearest to t, ties to the even code, at most 448."""
    t = np.asarray(t, np.float64)
    a = np.abs(t)
    lo = np.searchsorted(_MID, a, side="left")   # a tie goes to the lower code
    hi = np.searchsorted(_MID, a, side="right")  # a tie goes to the upper code
    code = np.where(lo % 2 == 0, lo, hi)
    code = np.where(np.isnan(t), 127, code)
    return (code + np.where(np.signbit(t) & ~np.isnan(t), 128, 0)).astype(np.uint8)


# ---- norm ----

def rms_norm(x, r, w, eps, offset):
    """(z, rstd, y) in float64 of float64 inputs (x or r may be None, w too)."""
    z = (0.0 if x is None else x) + (0.0 if r is None else r)
    rstd = 1.0 / np.sqrt((z * z).mean(axis=1) + eps)
    gain = (1.0 if w is None else w) + offset
    return z, rstd, z * rstd[:, None] * gain


def group_amax(y, group):
    T, d = y.shape
    g = group or d
    pad = np.zeros((T, -d % g))
    return np.abs(np.concatenate([y, pad], 1)).reshape(T, -1, g).max(axis=2)


def rms_norm_backward(dy, z, w, rstd, dres, offset):
    """(dz, dw, bound of |dz|'s terms, sum of |dw|'s terms) in float64."""
    zh = z * rstd[:, None]
    g = dy * ((1.0 if w is None else w) + offset)
    dz = rstd[:, None] * (g - zh * (g * zh).mean(axis=1, keepdims=True))
    size = rstd[:, None] * (np.abs(g) + np.abs(zh) * np.abs(g * zh).mean(axis=1, keepdims=True))
    if dres is not None:
        dz = dz + dres
        size = size + np.abs(dres)
    return dz, (dy * zh).sum(axis=0), size, np.abs(dy * zh).sum(axis=0)


# ---- AdamW, every operation rounded to float32 ----

def mix32(h):
    h = np.asarray(h, np.uint32)
    with np.errstate(over="ignore"):
        h = h ^ (h >> np.uint32(16))
        h = h * np.uint32(0x85EBCA6B)
        h = h ^ (h >> np.uint32(13))
        h = h * np.uint32(0xC2B2AE35)
        return h ^ (h >> np.uint32(16))


def words(seed: int, tensor: int, index: np.ndarray) -> np.ndarray:
    """The 32 random bits of a tensor's elements (index: int64)."""
    lo, hi = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    key = mix32(mix32(lo ^ ((0x9E3779B9 * (tensor + 1)) & 0xFFFFFFFF)) ^ np.uint32(hi))
    low = (index & 0xFFFFFFFF).astype(np.uint32)
    high = (((index >> 32) * 0x9E3779B9) & 0xFFFFFFFF).astype(np.uint32)
    return mix32(low ^ key ^ high)


def to_bf16(v: np.ndarray) -> np.ndarray:
    """float32 rounded to bfloat16 (nearest even), as float32."""
    b = v.astype(np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)
    return b.astype(np.uint32).view(np.float32)


def stochastic_bf16(v, bits16):
    b = v.astype(np.float32).view(np.uint32)
    return ((b + bits16.astype(np.uint32)) & np.uint32(0xFFFF0000)).view(np.float32)


def stochastic_e4m3(t, bits16):
    """Codes of t moved down or up: floor(|t| / step + u) step, without
    rounding on the way."""
    a = np.abs(t.astype(np.float64))
    _, e = np.frexp(a)
    e = np.maximum(e - 1, -6)
    k = np.floor(np.ldexp(a, 3 - e) + bits16.astype(np.float64) / 65536)
    v = np.minimum(np.ldexp(k, e - 3), 448.0)
    return e4m3_nearest(np.copysign(v, t))


def blocks(x):
    return np.concatenate([x, np.zeros(-len(x) % 128, x.dtype)]).reshape(-1, 128)


def quantise(x, bits16, floor):
    """(codes, scale) of a moment; bits16 None: to nearest."""
    f = np.float32
    s = np.maximum(np.abs(blocks(x)).max(axis=1) * (f(1) / f(448)), f(TINY)).astype(f)
    inv = (f(1) / s).astype(f)
    t = (blocks(x) * inv[:, None]).reshape(-1)[:len(x)].astype(f)
    codes = e4m3_nearest(t) if bits16 is None else stochastic_e4m3(t, bits16)
    if floor:
        codes = np.where((t > 0) & (codes == 0), 1, codes).astype(np.uint8)
    return codes, s


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, wd, step, gs=None, scale=None, seed=None, tensor=0,
          param_bf16=False, master=False):
    """One step of one tensor; p, g, m, v float32 arrays (m, v codes with
    ``scale`` [blocks, 2]).  Returns a dict of float32 arrays or codes."""
    f = np.float32
    if scale is not None:
        m = (blocks(E4M3[m].astype(f)) * scale[:, :1]).reshape(-1)[:len(p)].astype(f)
        v = (blocks(E4M3[v].astype(f)) * scale[:, 1:]).reshape(-1)[:len(p)].astype(f)
        v = v * v
    if gs is not None:
        g = g * f(gs)
    m = m * f(beta1) + g * f(1.0 - beta1)
    v = v * f(beta2) + (g * g) * f(1.0 - beta2)
    r = np.sqrt(v)
    root = f(1.0 / math.sqrt(1.0 - beta2 ** step))
    w = p * f(1.0 - lr * wd) - f(lr / (1.0 - beta1 ** step)) * (m / (r * root + f(eps)))
    assert w.dtype == f and r.dtype == f
    h = words(seed, tensor, np.arange(len(p), dtype=np.int64)) if seed is not None else None
    out = {"w": w}
    if param_bf16:
        if seed is not None and not master:
            out["p"] = stochastic_bf16(w, mix32(h ^ np.uint32(0x9E3779B9)) & np.uint32(0xFFFF))
        else:
            out["p"] = to_bf16(w)
    else:
        out["p"] = w
    if scale is None:
        out["m"], out["v"] = m, v
        return out
    out["m"], sm = quantise(m, None if h is None else h & np.uint32(0xFFFF), False)
    out["v"], sr = quantise(r, None if h is None else h >> np.uint32(16), True)
    out["scale"] = np.stack([sm, sr], 1)
    return out
