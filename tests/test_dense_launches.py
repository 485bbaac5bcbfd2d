"""What the dense block's entry points launch, on the CPU (launch_recorder.py)."""
import math
import random

import pytest

import launch_recorder as R
import sparse_tree_structured_amd as fff

F32, BF16, E4M3 = fff.DTYPE_F32, fff.DTYPE_BF16, fff.DTYPE_E4M3


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    lib = R.build(str(tmp_path_factory.mktemp("launches")))
    return lambda calls: R.record(lib, calls)


def shape(T, K, N, ty=BF16, **over):
    return dict(dict(T=T, K=K, N=N, dtype=ty, out_dtype=ty, act=0, save_dtype=ty, save_group=0, x_dtype=ty, x_group=0,
                     grad_dtype=F32), **over)


# Widths in eights and odd ones, narrow and wide.
WIDTHS = [(24, 40), (63, 65), (767, 2045), (4096, 8192), (4097, 8192), (8192, 4097), (4095, 11007), (8191, 8191),
          (65535, 1023), ((1 << 20) - 1, 127)]


@pytest.mark.parametrize("ty", [F32, BF16])
def test_no_rows(record, ty):
    """Gradients of no rows are zeros that a launch has to write, whatever the
    widths: a product over no rows copies nothing first."""
    calls = []
    for K, N in WIDTHS:
        for act, save, x in ((0, ty, ty), (2, E4M3, E4M3)):
            s = shape(0, K, N, ty, act=act, save_dtype=save, x_dtype=x)
            calls += [("fff_linear_backward", s, {}, False), ("fff_gated_backward", s, {}, False)]
    for (name, s, _, _), (status, kernels) in zip(calls, record(calls)):
        assert status == fff.SUCCESS, (name, s)
        dW = [k for k, _, _ in kernels if "product" in k]
        assert len(dW) == 1 and not [k for k, _, _ in kernels if "pad" in k or "split" in k], (name, s, kernels)


def test_a_captured_call_clears_the_word_of_its_planes(record):
    """Once, before any launch that writes or reads it; an eager call, whose
    number is its own, does not, and nor do products without planes."""
    sizes = {F32: (2048, 1024, 2048), BF16: (2048, 1024, 2048)}
    for ty, (T, K, N) in sizes.items():
        for small in (False, True):
            s = shape(48 if small else T, K, N, ty, act=2)
            calls = [(name, s, {}, captured) for name in R.ARGS for captured in (False, True)]
            for (name, _, _, captured), (status, kernels) in zip(calls, record(calls)):
                assert status == fff.SUCCESS
                names = [k for k, _, _ in kernels]
                cleared = [i for i, k in enumerate(names) if "clear_word" in k]
                assert cleared == ([0] if captured and ty == F32 and not small else []), (name, ty, small, names)


def test_every_shape_launches_or_is_refused(record):
    """Shapes over the whole range (widths up to 2^20, rows up to 2^31 - 1), operands
    aligned and not, outputs asked for and not: a launch never has no workgroups
    or more threads than HIP takes."""
    rng = random.Random(7)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    calls = []
    while len(calls) < 3000:
        ty, step, name = rng.choice([F32, BF16]), rng.choice([1, 8]), rng.choice(sorted(R.ARGS))
        T = rng.choice([0, 1, log(1, 64), log(64, 40000), log(1, 2 ** 31 - 1)])
        K, N = (step * log(1, (1 << 20) // step) for _ in range(2))
        if max(T * K, T * N, K * N) >= 1 << 40:
            continue
        back = "backward" in name
        save, x = (rng.choice([ty, E4M3]) for _ in range(2))
        s = shape(T, K, N, ty, act=rng.randrange(4), save_dtype=save,
                  save_group=rng.choice([32, 64, 128]) if save == E4M3 else 0, grad_dtype=rng.choice([ty, F32]))
        if back:
            s.update(x_dtype=x, x_group=rng.choice([0, 32, 64, 128]) if x == E4M3 else 0)
        elif name == "fff_linear":
            s.update(out_dtype=rng.choice([ty, F32]))
        p = {k: (1 << 40) + 4 for k in ("x", "W", "Wg", "Wu", "dy", "dh") if rng.random() < 0.2}
        may_be_none = ["dx", "dbias"] if back else ["bias", "residual", "pre", "gate", "up"]
        p.update({k: 0 for k in may_be_none if rng.random() < 0.3})
        if back and rng.random() < 0.3:
            p.update(dW=0, dWg=0, dWu=0)
        calls.append((name, s, p, rng.random() < 0.2))
    for call, (status, _) in zip(calls, record(calls)):
        assert status in (fff.SUCCESS, fff.ERROR_NOT_SUPPORTED), call
