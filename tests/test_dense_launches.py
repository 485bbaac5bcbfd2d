"""What the dense block's entry points launch, on the CPU (launch_recorder.py)."""
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
