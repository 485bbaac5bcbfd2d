"""The norm's and the optimiser's host-side checks, on the CPU: the C entry
points return the documented codes before any HIP call, and the binding
raises ValueError for wrong tensors."""
import ctypes
import math

import pytest
import torch

import sparse_tree_structured_amd as fff

FAKE, ODD = 0x10000, 0x10001  # never dereferenced: validation fails first
F32, BF16, E4M3 = fff.DTYPE_F32, fff.DTYPE_BF16, fff.DTYPE_E4M3
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    return fff.load_library()


def norm_shape(**over):
    f = dict(T=4, d=64, dtype=BF16, stream_dtype=F32, out_dtype=BF16, group=0, eps=1e-6, weight_offset=0.0)
    f.update(over)
    return fff.NormShape(**f)


def norm(lib, shape=None, **p):
    a = dict(x=FAKE, r=FAKE, w=FAKE, y=FAKE, s=FAKE, z=FAKE, rstd=FAKE)
    a.update(p)
    return lib.fff_rms_norm(shape or norm_shape(), a["x"], a["r"], a["w"], a["y"], a["s"], a["z"], a["rstd"], None)


BAD_SHAPES = [
    (dict(dtype=7), fff.ERROR_NOT_SUPPORTED), (dict(dtype=E4M3), fff.ERROR_NOT_SUPPORTED),
    (dict(stream_dtype=E4M3), fff.ERROR_NOT_SUPPORTED),
    (dict(dtype=F32, stream_dtype=BF16, out_dtype=F32), fff.ERROR_NOT_SUPPORTED),
    (dict(d=32769), fff.ERROR_NOT_SUPPORTED), (dict(d=0), fff.ERROR_INVALID_VALUE),
    (dict(T=-1), fff.ERROR_INVALID_VALUE), (dict(T=1 << 31), fff.ERROR_INVALID_VALUE),
    (dict(T=(1 << 31) - 1, d=4096), fff.ERROR_INVALID_VALUE),
    (dict(eps=-1.0), fff.ERROR_INVALID_VALUE), (dict(eps=math.nan), fff.ERROR_INVALID_VALUE),
    (dict(weight_offset=math.inf), fff.ERROR_INVALID_VALUE),
]


@pytest.mark.parametrize("over,code", BAD_SHAPES)
def test_norm_shape(lib, over, code):
    assert norm(lib, norm_shape(**over)) == code
    n = ctypes.c_size_t()
    assert lib.fff_rms_norm_backward_workspace_size(norm_shape(**over), ctypes.byref(n)) == code
    assert lib.fff_rms_norm_backward(norm_shape(**over), *[FAKE] * 9, 1 << 30, None) == code


def test_norm_output_type_and_group(lib):
    assert norm(lib, norm_shape(out_dtype=F32)) == fff.ERROR_NOT_SUPPORTED
    assert norm(lib, norm_shape(out_dtype=9)) == fff.ERROR_NOT_SUPPORTED
    for group in (-32, 1, 16, 96, 256):
        assert norm(lib, norm_shape(out_dtype=E4M3, group=group)) == fff.ERROR_INVALID_VALUE
    assert norm(lib, norm_shape(group=32)) == fff.ERROR_INVALID_VALUE


@pytest.mark.parametrize("over", [dict(x=None, r=None), dict(y=None), dict(x=ODD), dict(r=FAKE + 2),
                                  dict(w=ODD), dict(y=ODD), dict(z=FAKE + 2), dict(rstd=FAKE + 2)])
def test_norm_pointers(lib, over):
    assert norm(lib, **over) == fff.ERROR_INVALID_VALUE


def test_norm_scale_pointer(lib):
    s = norm_shape(out_dtype=E4M3)
    assert norm(lib, s, s=None) == fff.ERROR_INVALID_VALUE
    assert norm(lib, s, s=FAKE + 2) == fff.ERROR_INVALID_VALUE


def test_no_rows_touches_nothing(lib):
    assert lib.fff_rms_norm(norm_shape(T=0), *[None] * 8) == fff.SUCCESS
    assert lib.fff_rms_norm_backward(norm_shape(T=0), *[None] * 9, 0, None) == fff.SUCCESS
    n = ctypes.c_size_t(5)
    assert lib.fff_rms_norm_backward_workspace_size(norm_shape(T=0), ctypes.byref(n)) == 0 and n.value == 0


def test_norm_backward_pointers_and_workspace(lib):
    s = norm_shape(T=30000)
    need = ctypes.c_size_t()
    assert lib.fff_rms_norm_backward_workspace_size(s, ctypes.byref(need)) == fff.SUCCESS
    assert need.value >= 64 * 4 and lib.fff_rms_norm_backward_workspace_size(s, None) == fff.ERROR_INVALID_VALUE
    names = ["dy", "z", "w", "rstd", "dres", "dz", "dx", "dw", "ws"]

    def call(n=1 << 30, **over):
        return lib.fff_rms_norm_backward(s, *[over.get(k, FAKE) for k in names], n, None)

    for over in (dict(dy=None), dict(z=None), dict(rstd=None), dict(dz=None), dict(dy=ODD), dict(z=FAKE + 2),
                 dict(w=ODD), dict(rstd=ODD), dict(dres=FAKE + 2), dict(dz=FAKE + 2), dict(dx=ODD), dict(dw=ODD),
                 dict(ws=FAKE + 128)):
        assert call(**over) == fff.ERROR_INVALID_VALUE, over
    assert call(ws=None) == fff.ERROR_WORKSPACE and call(n=need.value - 1) == fff.ERROR_WORKSPACE


def entry(**over):
    f = dict(param=FAKE, master=None, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, scale=None, n=10,
             param_dtype=F32, grad_dtype=F32, lr_scale=1.0, weight_decay=0.0)
    f.update(over)
    return fff.AdamwTensor(**f)


def config(**over):
    f = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, state_dtype=F32)
    f.update(over)
    return fff.AdamwConfig(**f)


def step(lib, e=None, c=None, count=1):
    return lib.fff_adamw_step(c or config(), (fff.AdamwTensor * 1)(e or entry()), count, None)


@pytest.mark.parametrize("over", [dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
                                  dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.inf),
                                  dict(step=0), dict(grad_scale=ODD)])
def test_adamw_config(lib, over):
    assert step(lib, c=config(**over)) == fff.ERROR_INVALID_VALUE


def test_adamw_state_type(lib):
    assert step(lib, c=config(state_dtype=BF16)) == fff.ERROR_NOT_SUPPORTED
    assert step(lib, c=config(state_dtype=E4M3)) == fff.ERROR_INVALID_VALUE  # no scale
    assert step(lib, entry(scale=FAKE + 4), config(state_dtype=E4M3)) == fff.ERROR_INVALID_VALUE


@pytest.mark.parametrize("over,code", [
    (dict(param=None), 1), (dict(grad=None), 1), (dict(exp_avg=None), 1), (dict(exp_avg_sq=None), 1),
    (dict(param=FAKE + 2), 1), (dict(grad=ODD), 1), (dict(exp_avg=FAKE + 2), 1), (dict(n=-1), 1),
    (dict(n=(1 << 34) + 1), 1), (dict(grad=1 << 48), 1), (dict(param=(1 << 63) + FAKE), 1), (dict(lr_scale=math.nan), 1), (dict(weight_decay=math.inf), 1),
    (dict(master=FAKE), 2), (dict(param_dtype=BF16, master=FAKE + 2), 1), (dict(param_dtype=E4M3), 2),
    (dict(grad_dtype=E4M3), 2), (dict(grad_dtype=5), 2)])
def test_adamw_tensor(lib, over, code):
    assert step(lib, entry(**over)) == code
    two = (fff.AdamwTensor * 2)(entry(n=0), entry(**over))  # found wherever it is in the list
    assert lib.fff_adamw_step(config(), two, 2, None) == code


def test_adamw_nothing_to_do(lib):
    assert lib.fff_adamw_step(config(), None, 0, None) == fff.SUCCESS
    assert step(lib, entry(n=0, param=None, grad=None, exp_avg=None, exp_avg_sq=None)) == fff.SUCCESS
    assert lib.fff_adamw_step(config(), None, 1, None) == fff.ERROR_INVALID_VALUE
    assert lib.fff_adamw_step(config(), None, -1, None) == fff.ERROR_INVALID_VALUE
    assert lib.fff_adamw_step(None, None, 0, None) == fff.ERROR_INVALID_VALUE


def test_grad_norm(lib):
    t = (fff.AdamwTensor * 1)(entry(n=1000000))
    n = ctypes.c_size_t()
    assert lib.fff_grad_norm_workspace_size(t, 1, ctypes.byref(n)) == fff.SUCCESS and n.value >= 8
    assert lib.fff_grad_norm_workspace_size(t, 1, None) == fff.ERROR_INVALID_VALUE

    def call(tensors=t, limit=1.0, out=FAKE, ws=FAKE, size=1 << 20):
        return lib.fff_grad_norm(tensors, 1, limit, out, ws, size, None)

    for limit in (0.0, -1.0, math.nan):
        assert call(limit=limit) == fff.ERROR_INVALID_VALUE
    assert call(out=None) == fff.ERROR_INVALID_VALUE and call(out=ODD) == fff.ERROR_INVALID_VALUE
    assert call(ws=None) == fff.ERROR_WORKSPACE and call(size=n.value - 1) == fff.ERROR_WORKSPACE
    assert call(ws=FAKE + 8) == fff.ERROR_INVALID_VALUE
    assert call((fff.AdamwTensor * 1)(entry(grad=None))) == fff.ERROR_INVALID_VALUE
    assert call((fff.AdamwTensor * 1)(entry(grad_dtype=E4M3))) == fff.ERROR_NOT_SUPPORTED


# ---- the binding ----

B = torch.bfloat16
X, W = torch.zeros(4, 64, dtype=B), torch.zeros(64, dtype=B)


@pytest.mark.parametrize("x,kw,name", [
    (torch.zeros(2, 2, 8), {}, "x"),
    (X, dict(weight=torch.zeros(63, dtype=B)), "weight"),
    (X, dict(weight=W, residual=torch.zeros(3, 64)), "residual"),
    (X.float(), dict(weight=W, residual=X), "x must be"),
    (X.t().contiguous().t(), dict(weight=W), "contiguous"),
    (X, dict(weight=W, y=torch.zeros(4, 64)), "y must be"),
    (X, dict(weight=W, out_dtype=F8, y=X), "y must be"),
    (X, dict(weight=W), "GPU"),
])
def test_rms_norm_rejects(x, kw, name):
    with pytest.raises(ValueError, match=name):
        fff.rms_norm(x, **kw)
    with pytest.raises(TypeError):
        fff.rms_norm(X.half())


@pytest.mark.parametrize("over,name", [
    (dict(z=torch.zeros(4, 63)), "z"), (dict(rstd=torch.zeros(3)), "rstd"),
    (dict(rstd=torch.zeros(4, dtype=B)), "rstd"), (dict(weight=W.float()), "weight"),
    (dict(dresidual=torch.zeros(4, 64)), "dresidual"), ({}, "GPU")])
def test_rms_norm_backward_rejects(over, name):
    a = dict(dy=X, z=X, weight=W, rstd=torch.zeros(4))
    a.update(over)
    with pytest.raises(ValueError, match=name):
        fff.rms_norm_backward(a.pop("dy"), a.pop("z"), a.pop("weight"), a.pop("rstd"), **a)


def test_tables_reject():
    p = [torch.zeros(10)]
    with pytest.raises(ValueError, match="GPU"):
        fff.adamw_table(p, p, p, p)
    with pytest.raises(ValueError, match="GPU"):
        fff.grad_table(p)
    with pytest.raises(ValueError, match="one entry for each"):
        fff.adamw_table(p, p + p, p, p)
    with pytest.raises(ValueError, match="exp_avg must be"):
        fff.adamw_table(p, p, [torch.zeros(10, dtype=B)], p)
    with pytest.raises(ValueError, match="at least one"):
        fff.adamw_table([], [], [], [])
    with pytest.raises(ValueError, match="at least one"):
        fff.grad_table([])
    with pytest.raises(ValueError, match="bits"):
        fff.adamw_state(p, bits=16)


def test_adamw_state_shapes():
    m, v, s = fff.adamw_state([torch.zeros(3, 100), torch.zeros(128)], bits=8)
    assert m[0].dtype == F8 and v[0].shape == (3, 100) and [tuple(t.shape) for t in s] == [(3, 2), (1, 2)]
    m, v, s = fff.adamw_state([torch.zeros(3, dtype=B)])
    assert m[0].dtype == torch.float32 and s is None
