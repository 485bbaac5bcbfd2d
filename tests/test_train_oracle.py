"""The numpy forms that the norm's and the optimiser's GPU tests compare with,
checked on the CPU against what the formulas fix."""
import math

import numpy as np
import pytest
import torch

import train_oracle as O


def test_e4m3_values_and_rounding():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(codes[:127], O.E4M3[:127]) and np.isnan(codes[127])
    rng = np.random.default_rng(0)
    t = np.concatenate([rng.uniform(-448, 448, 20000), rng.normal(size=20000) * 0.01,
                        O._MID, -O._MID, O._POS, [0.0, -0.0]]).astype(np.float32)
    want = torch.from_numpy(t).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_nearest(t), want)


def test_stochastic_rounding_brackets_and_keeps_the_mean():
    rng = np.random.default_rng(1)
    t = (rng.uniform(-448, 448, 2000) * 10.0 ** rng.uniform(-6, 0, 2000)).astype(np.float32)
    bits = np.arange(0, 65536, 64)  # u on an even grid: the mean is exact to 64 / 2^16
    got = np.stack([O.E4M3[O.stochastic_e4m3(t, np.full(t.shape, b))] for b in bits])
    a = np.abs(t)
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    assert (np.abs(got - t) < step).all()
    assert (np.abs(got.mean(axis=0) - t) <= step * 64 / 65536 + 1e-12).all()


def test_stochastic_bf16_brackets_and_keeps_the_mean():
    rng = np.random.default_rng(2)
    v = rng.normal(size=500).astype(np.float32)
    got = np.stack([O.stochastic_bf16(v, np.full(v.shape, b)) for b in range(0, 65536, 64)]).astype(np.float64)
    step = 2.0 ** (np.floor(np.log2(np.abs(v.astype(np.float64)))) - 7)
    assert (np.abs(got - v) < step).all()
    assert (np.abs(got.mean(axis=0) - v) <= step * 64 / 65536).all()


def test_words_differ_by_seed_tensor_and_high_index():
    i = np.arange(1000, dtype=np.int64)
    a = O.words(5, 0, i)
    for b in (O.words(6, 0, i), O.words(5, 1, i), O.words(5 + (1 << 40), 0, i), O.words(5, 0, i + (1 << 32))):
        assert (a != b).mean() > 0.99
    assert abs((a & 0xFFFF).mean() / 65536 - 0.5) < 0.05 and abs((a >> 16).mean() / 65536 - 0.5) < 0.05


@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm_gradient_against_differences(offset):
    rng = np.random.default_rng(3)
    T, d, eps = 5, 12, 1e-6
    z, w = rng.normal(size=(T, d)), rng.normal(size=d)
    dy, dres = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def f(z, w):
        return (O.rms_norm(None, z, w, eps, offset)[2] * dy).sum() + (z * dres).sum()

    rstd = O.rms_norm(None, z, w, eps, offset)[1]
    dz, dw, _, _ = O.rms_norm_backward(dy, z, w, rstd, dres, offset)
    h = 1e-5
    for i in range(T):
        for j in range(d):
            e = np.zeros((T, d))
            e[i, j] = h
            assert abs((f(z + e, w) - f(z - e, w)) / (2 * h) - dz[i, j]) < 1e-7
    for j in range(d):
        e = np.zeros(d)
        e[j] = h
        assert abs((f(z, w + e) - f(z, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_adamw_against_torch():
    """torch's own AdamW on the CPU, in 64 bits, over a few steps."""
    rng = np.random.default_rng(4)
    n, kw = 300, dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1)
    p = rng.normal(size=n).astype(np.float32)
    q = torch.nn.Parameter(torch.from_numpy(p.astype(np.float64)))
    opt = torch.optim.AdamW([q], lr=kw["lr"], betas=(kw["beta1"], kw["beta2"]), eps=kw["eps"],
                            weight_decay=kw["wd"])
    m = v = np.zeros(n, np.float32)
    for step in range(1, 6):
        g = rng.normal(size=n).astype(np.float32)
        o = O.adamw(p, g, m, v, step=step, **kw)
        p, m, v = o["p"], o["m"], o["v"]
        q.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
    # five steps of a dozen roundings each on values near 1
    assert np.abs(p - q.detach().numpy()).max() < 5 * 12 * O.U32 * 4


def test_eight_bit_state_moves_only_stochastically():
    """A second moment whose gradient vanished decays by 0.1 % a step: nearest
    codes stay for ever, stochastic ones follow the decay on average."""
    n, steps, beta2 = 128 * 64, 200, 0.999
    r0 = np.ones(n, np.float32)
    r0[::128] = 4.0  # every block's largest, kept up by its gradient
    g = np.where(r0 == 4.0, 4.0, 0.0).astype(np.float32)
    end = {}
    for seed in (None, 11):
        codes, scale = O.quantise(r0, None, True)
        m, sc = np.zeros(n, np.uint8), np.stack([np.full(64, O.TINY, np.float32), scale], 1)
        for step in range(1, steps + 1):
            o = O.adamw(np.zeros(n, np.float32), g, m, codes, lr=0.0, beta1=0.0, beta2=beta2, eps=1e-8,
                        wd=0.0, step=step, scale=sc, seed=None if seed is None else seed + step)
            m, codes, sc = o["m"], o["v"], o["scale"]
        r = (O.blocks(O.E4M3[codes]) * sc[:, 1:])
        end[seed] = r.reshape(-1)[np.arange(n) % 128 != 0].mean()
    assert end[None] > 0.99
    assert abs(end[11] - math.sqrt(beta2 ** steps)) < 0.02
