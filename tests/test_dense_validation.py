"""The dense block's host-side checks, on the CPU: the C entry points return
the documented codes before any HIP call, and the binding refuses wrong
arguments."""
import ctypes

import pytest
import torch

import sparse_tree_structured_amd as fff

FAKE, ODD = 0x10000, 0x10001  # never dereferenced: validation fails first
F32, BF16, E4M3 = fff.DTYPE_F32, fff.DTYPE_BF16, fff.DTYPE_E4M3
BAD, NOT, WS = fff.ERROR_INVALID_VALUE, fff.ERROR_NOT_SUPPORTED, fff.ERROR_WORKSPACE
B, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    return fff.load_library()


def shape(**over):
    f = dict(T=8, K=64, N=128, dtype=BF16, out_dtype=BF16, act=0, save_dtype=BF16, save_group=0,
             x_dtype=BF16, x_group=0, grad_dtype=F32)
    f.update(over)
    return fff.DenseShape(**f)


ARGS = {
    "fff_linear": ["x", "W", "bias", "residual", "y", "pre", "pre_scale", "ws"],
    "fff_linear_backward": ["dy", "x", "x_scale", "W", "pre", "pre_scale", "dx", "dW", "dbias", "ws"],
    "fff_gated": ["x", "Wg", "Wu", "h", "gate", "gate_scale", "up", "up_scale", "ws"],
    "fff_gated_backward": ["dh", "x", "x_scale", "Wg", "Wu", "gate", "gate_scale", "up", "up_scale", "dx",
                           "dWg", "dWu", "h", "ws"],
}


def call(lib, name, s, n=1 << 62, **over):
    return getattr(lib, name)(s, *[over.get(k, FAKE) for k in ARGS[name]], n, None)


SHAPES = [
    (dict(dtype=7), NOT), (dict(dtype=E4M3), NOT), (dict(T=-1), BAD), (dict(T=1 << 31), BAD),
    (dict(K=0), BAD), (dict(N=0), BAD), (dict(K=-5), BAD), (dict(K=(1 << 20) + 1), NOT),
    (dict(N=(1 << 20) + 1), NOT), (dict(T=1 << 30, K=1 << 10), BAD), (dict(T=1 << 30, N=1 << 10), BAD),
    (dict(K=1 << 20, N=1 << 20), BAD), (dict(act=-1), BAD), (dict(act=4), BAD), (dict(save_dtype=F32), NOT),
    (dict(save_dtype=9), NOT), (dict(save_group=32), BAD), (dict(save_dtype=E4M3, save_group=96), BAD),
    (dict(save_dtype=E4M3, save_group=-32), BAD), (dict(T=(1 << 31) - 1), NOT),
]
FORWARD = [(dict(out_dtype=E4M3), NOT), (dict(dtype=F32, save_dtype=F32, out_dtype=BF16), NOT),
           (dict(save_dtype=E4M3, save_group=0), BAD)]
BACKWARD = [(dict(x_dtype=F32), NOT), (dict(x_group=64), BAD), (dict(x_dtype=E4M3, x_group=16), BAD),
            (dict(grad_dtype=E4M3), NOT), (dict(dtype=F32, save_dtype=F32, x_dtype=F32, grad_dtype=BF16), NOT)]


@pytest.mark.parametrize("name", ARGS)
def test_shapes(lib, name):
    n = ctypes.c_size_t()
    for over, code in SHAPES + (BACKWARD if "backward" in name else FORWARD):
        assert call(lib, name, shape(**over)) == code, over
        assert getattr(lib, name + "_workspace_size")(shape(**over), ctypes.byref(n)) == code, over
    assert getattr(lib, name + "_workspace_size")(shape(), None) == BAD
    assert getattr(lib, name + "_workspace_size")(None, ctypes.byref(n)) == BAD


def test_gated_output_type(lib):
    assert call(lib, "fff_gated", shape(out_dtype=F32)) == NOT


@pytest.mark.parametrize("name", ARGS)
def test_pointers(lib, name):
    e = E4M3 if "backward" in name else BF16
    s = shape(act=1, save_dtype=E4M3, save_group=32, x_dtype=e, x_group=32 if e == E4M3 else 0)
    optional = {"bias", "residual", "pre", "dx", "dW", "dbias", "h", "gate", "up"}
    if "backward" in name:
        optional -= {"pre", "gate", "up"}
    if name == "fff_gated":
        optional -= {"h"}
    bytes_ok = {"pre", "gate", "up"} | ({"x"} if e == E4M3 else set())  # codes have no alignment
    for k in ARGS[name]:
        if k == "ws":
            continue
        if k not in bytes_ok:
            assert call(lib, name, s, **{k: ODD}) == BAD, k
        if k not in optional and k not in ("dWg", "dWu"):
            assert call(lib, name, s, **{k: None}) == BAD, k
    if name == "fff_gated_backward":
        assert call(lib, name, s, dWg=None) == BAD and call(lib, name, s, dWu=None) == BAD


@pytest.mark.parametrize("name", ARGS)
def test_workspace(lib, name):
    s = shape(T=4, K=4096, N=64, act=1)
    need = ctypes.c_size_t()
    assert getattr(lib, name + "_workspace_size")(s, ctypes.byref(need)) == fff.SUCCESS
    if need.value:
        assert call(lib, name, s, n=need.value - 1) == WS and call(lib, name, s, ws=None) == WS
    assert call(lib, name, s, ws=FAKE + 128) == BAD


def test_nothing_to_do_touches_nothing(lib):
    s = shape(T=0)
    for name in ("fff_linear", "fff_gated"):
        assert getattr(lib, name)(s, *[None] * len(ARGS[name]), 0, None) == fff.SUCCESS
    for name in ("fff_linear_backward", "fff_gated_backward"):
        for T in (0, 8):
            assert getattr(lib, name)(shape(T=T), *[None] * len(ARGS[name]), 0, None) == fff.SUCCESS
    n = ctypes.c_size_t(5)
    for name in ARGS:
        assert getattr(lib, name + "_workspace_size")(s, ctypes.byref(n)) == 0 and n.value == 0


def test_checkpoint_arguments(lib):
    for f in (lib.fff_checkpoint_save, lib.fff_checkpoint_load):
        ok = dict(T=4, d=64, dtype=BF16, group=32)
        for over, code in ((dict(dtype=E4M3), NOT), (dict(T=-1), BAD), (dict(T=1 << 31), BAD), (dict(d=0), BAD),
                           (dict(d=(1 << 20) + 1), NOT), (dict(T=1 << 30, d=1 << 10), BAD), (dict(group=16), BAD),
                           (dict(group=-32), BAD), (dict(group=256), BAD)):
            a = {**ok, **over}
            assert f(a["T"], a["d"], a["dtype"], a["group"], FAKE, FAKE, FAKE, None) == code, over
        assert f(0, 64, BF16, 32, None, None, None, None) == fff.SUCCESS
        for ptrs in ([None, FAKE, FAKE], [FAKE, None, FAKE], [FAKE, FAKE, None], [FAKE, FAKE, ODD]):
            assert f(4, 64, BF16, 32, *ptrs, None) == BAD
    assert lib.fff_checkpoint_save(4, 64, BF16, 32, ODD, FAKE, FAKE, None) == BAD
    assert lib.fff_checkpoint_load(4, 64, BF16, 32, FAKE, FAKE, ODD, None) == BAD


# ---- the binding: a stub in the library's place records what reaches it ----

class Library:
    def __init__(self):
        self.calls = []
        real = fff.load_library()
        self.fff_status_string = real.fff_status_string
        for name in ARGS:
            setattr(self, name + "_workspace_size", getattr(real, name + "_workspace_size"))

    def __getattr__(self, name):
        def f(*args):
            self.calls.append((name, args))
            return fff.SUCCESS
        return f


@pytest.fixture
def stub(monkeypatch):
    s = Library()
    monkeypatch.setattr(fff, "_lib", s)
    monkeypatch.setattr(fff, "_here", lambda rt, t, stream: 0)
    fff._dense.cache_clear()
    yield s
    fff._dense.cache_clear()


def z(*s, dtype=B):
    return torch.zeros(*s, dtype=dtype)


def test_what_reaches_the_library(stub):
    o = fff.linear(z(4, 64), z(64, 128), z(128), residual=z(4, 128, dtype=torch.float32), act="gelu",
                   save="e4m3", group=32)
    name, (s, *p) = stub.calls.pop()
    assert name == "fff_linear" and (s.T, s.K, s.N, s.dtype, s.out_dtype, s.act) == (4, 64, 128, BF16, F32, 1)
    assert (s.save_dtype, s.save_group) == (E4M3, 32) and o.y.dtype is torch.float32
    assert o.pre.codes.shape == (4, 128) and o.pre.scale.shape == (4, 4) and o.pre.group == 32
    assert p[4] == o.y.data_ptr() and p[5] == o.pre.codes.data_ptr() and p[6] == o.pre.scale.data_ptr()
    x8 = fff.Checkpoint(z(4, 64, dtype=F8), z(4, 1, dtype=torch.float32), 0)
    b = fff.linear_backward(z(4, 128), x8, z(64, 128), act="gelu", pre=o.pre, want_dx=False, grad_dtype=B)
    name, (s, *p) = stub.calls.pop()
    assert (s.x_dtype, s.x_group, s.save_dtype, s.save_group, s.grad_dtype) == (E4M3, 0, E4M3, 32, BF16)
    assert b.dx is None and b.dbias is None and b.dW.dtype is B and p[6] == 0 and p[7] == b.dW.data_ptr()
    g = fff.gated(z(4, 64), z(64, 128), z(64, 128), act="relu", save="same")
    name, (s, *p) = stub.calls.pop()
    assert name == "fff_gated" and s.act == 3 and g.gate.dtype is B and g.up.data_ptr() == p[6]
    r = fff.gated_backward(z(4, 128), None, z(64, 128), z(64, 128), g.gate, g.up, want_dW=False, want_h=True)
    name, (s, *p) = stub.calls.pop()
    assert p[10] == p[11] == 0 and r.dW_gate is None and p[12] == r.h.data_ptr() and p[1] == 0
    c = fff.checkpoint(z(4, 300), 64)
    assert c.scale.shape == (4, 5) and stub.calls.pop()[1][:4] == (4, 300, BF16, 64)
    assert fff.restore(c, torch.float32).dtype is torch.float32


REFUSED = [
    lambda: fff.linear(z(4, 64), z(32, 128)), lambda: fff.linear(z(4, 64), z(64, 128), z(64)),
    lambda: fff.linear(z(64), z(64, 128)), lambda: fff.linear(z(4, 64), z(64, 128, dtype=torch.float32)),
    lambda: fff.linear(z(64, 4).t(), z(64, 128)), lambda: fff.linear(z(4, 64), z(128, 64).t()),
    lambda: fff.linear(z(4, 64), z(64, 128), act="tanh"), lambda: fff.linear(z(4, 64), z(64, 128), save="bf16"),
    lambda: fff.linear(z(4, 64), z(64, 128), residual=z(4, 64)),
    lambda: fff.linear(z(4, 64), z(64, 128), residual=z(4, 128), out_dtype=torch.float32),
    lambda: fff.linear(z(4, 64), z(64, 128), y=z(4, 128), out_dtype=torch.float32),
    lambda: fff.linear(z(4, 64), z(64, 128), workspace=z(10)),
    lambda: fff.linear_backward(z(4, 128), None, z(64, 128)),
    lambda: fff.linear_backward(z(4, 128), z(4, 64), z(64, 128), act="silu"),
    lambda: fff.linear_backward(z(4, 128), z(4, 32), z(64, 128)),
    lambda: fff.linear_backward(z(4, 128), z(4, 64), z(64, 128), dW=z(64, 128), grad_dtype=torch.float32),
    lambda: fff.linear_backward(z(4, 128), fff.Checkpoint(z(4, 64, dtype=F8), z(4, 2, dtype=torch.float32), 64),
                                z(64, 128)),
    lambda: fff.linear_backward(z(4, 128), fff.Checkpoint(z(4, 64), z(4, 1, dtype=torch.float32), 64),
                                z(64, 128)),
    lambda: fff.linear_backward(z(4, 128), fff.Checkpoint(z(4, 64, dtype=F8), z(4, 4, dtype=torch.float32), 16),
                                z(64, 128)),
    lambda: fff.gated(z(4, 64), z(64, 128), z(64, 64)),
    lambda: fff.gated_backward(z(4, 128), None, z(64, 128), z(64, 128), z(4, 128), z(4, 128)),
    lambda: fff.gated_backward(z(4, 128), z(4, 64), z(64, 128), z(64, 128), z(4, 128),
                               fff.Checkpoint(z(4, 128, dtype=F8), z(4, 1, dtype=torch.float32), 128)),
    lambda: fff.gated_backward(z(4, 128), z(4, 64), z(64, 128), z(64, 128), z(4, 128), z(4, 128),
                               dW_up=z(64, 128)),
    lambda: fff.checkpoint(z(4)), lambda: fff.checkpoint(z(4, 64), codes=z(4, 64)),
    lambda: fff.checkpoint(z(4, 64), 32, scale=z(4, 1, dtype=torch.float32)),
    lambda: fff.restore(fff.Checkpoint(z(4, 64, dtype=F8), z(4, 2), 32)),
]


@pytest.mark.parametrize("k", range(len(REFUSED)))
def test_refused_by_the_binding(stub, k):
    with pytest.raises(ValueError):
        REFUSED[k]()
    assert not stub.calls


def test_types_and_sizes_that_are_not_supported(stub):
    with pytest.raises(TypeError):
        fff.linear(z(4, 64, dtype=torch.float16), z(64, 128, dtype=torch.float16))
    with pytest.raises(TypeError):
        fff.checkpoint(z(4, 64, dtype=torch.float64))
    for wide in ((1 << 20) + 1, (1 << 32) + 64):
        x, W = torch.empty(4, wide, dtype=B, device="meta"), torch.empty(wide, 8, dtype=B, device="meta")
        for f in (lambda: fff.linear(x, W), lambda: fff.gated(x, W, W), lambda: fff.checkpoint(x, 64)):
            with pytest.raises(fff.FFFError) as e:
                f()
            assert e.value.status == NOT
    for group in (0, 16, (1 << 32) + 32):
        with pytest.raises(fff.FFFError) as e:
            fff.linear(z(4, 64), z(64, 128), save="e4m3", group=group)
        assert e.value.status == BAD
    for group in (16, -32, (1 << 32) + 32):
        with pytest.raises(fff.FFFError):
            fff.checkpoint(z(4, 64), group)
    assert not stub.calls


def test_tensors_must_be_on_a_gpu():
    for f in (lambda: fff.linear(z(4, 64), z(64, 128)), lambda: fff.gated(z(4, 64), z(64, 128), z(64, 128)),
              lambda: fff.checkpoint(z(4, 64)), lambda: fff.linear_backward(z(4, 128), z(4, 64), z(64, 128))):
        with pytest.raises(ValueError):
            f()
