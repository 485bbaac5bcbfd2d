"""What the binding of the norm and the optimiser hands to the library, on the
CPU: the library is a stub that records its arguments, and tensors are on the
CPU or have no memory at all."""
import pytest
import torch

import sparse_tree_structured_amd as fff

B, F8 = torch.bfloat16, torch.float8_e4m3fn


class Library:
    """Records the descriptor of every call."""

    def __init__(self):
        self.shapes = []
        self.fff_status_string = fff.load_library().fff_status_string

    def __getattr__(self, name):
        def call(shape, *args):
            self.shapes.append(shape)
            return fff.SUCCESS
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(fff, "_lib", lib)
    monkeypatch.setattr(fff, "_here", lambda rt, t, stream: 0)
    fff._norm_shape.cache_clear()
    fff.rms_norm_backward_workspace_size.cache_clear()
    yield lib
    fff._norm_shape.cache_clear()
    fff.rms_norm_backward_workspace_size.cache_clear()


@pytest.mark.parametrize("group", [(1 << 32) + 32, (1 << 32), -(1 << 32) + 64, 1 << 31, -(1 << 31) - 1])
def test_a_group_beyond_its_field_is_refused(lib, group):
    """In 32 bits the first would be a group of 32 beside one scale a row."""
    with pytest.raises(fff.FFFError) as e:
        fff.rms_norm(torch.zeros(4, 256, dtype=B), out_dtype=F8, group=group)
    assert e.value.status == fff.ERROR_INVALID_VALUE and not lib.shapes


@pytest.mark.parametrize("d", [1 << 31, (1 << 32) + 64])
def test_a_width_beyond_its_field_is_refused(lib, d):
    """In 32 bits the second would be a width of 64.  The tensors have no
    memory."""
    x, f = (torch.empty(1, d, dtype=t, device="meta") for t in (B, torch.float32))
    w, rstd = torch.empty(d, dtype=B, device="meta"), torch.empty(1, device="meta")
    for call in (lambda: fff.rms_norm(x, w), lambda: fff.rms_norm(x, w, residual=f),
                 lambda: fff.rms_norm(f, w, out_dtype=F8, group=32),
                 lambda: fff.rms_norm_backward(x, f, w, rstd),
                 lambda: fff.rms_norm_backward(x, f, w, rstd, want_dweight=False),
                 lambda: fff.rms_norm_backward_workspace_size(1, d, fff.DTYPE_BF16, fff.DTYPE_F32)):
        with pytest.raises(fff.FFFError) as e:
            call()
        assert e.value.status == fff.ERROR_NOT_SUPPORTED
    assert not lib.shapes


def test_what_fits_reaches_the_library_as_it_is(lib):
    fff.rms_norm(torch.zeros(4, 300, dtype=B), out_dtype=F8, group=64, eps=0.5, weight_offset=1.0)
    s = lib.shapes.pop()
    assert (s.T, s.d, s.group, s.eps, s.weight_offset) == (4, 300, 64, 0.5, 1.0)


def test_a_group_that_fits_its_field_is_the_librarys_to_refuse():
    """(-32, 96 and 256 never reach a kernel: the C entry point returns first.)"""
    for group in (-32, 96, 256):
        s = fff._norm_shape(4, 300, fff.DTYPE_BF16, fff.DTYPE_BF16, fff.DTYPE_E4M3, group, 1e-6, 0.0)
        assert s.group == group
        assert fff.load_library().fff_rms_norm(s, *[0x10000] * 7, None) == fff.ERROR_INVALID_VALUE


# ---- the optimiser's table ----

@pytest.fixture
def on_cpu(monkeypatch):
    """Tables of CPU tensors: nothing steps them."""
    def flat(t, n, dtypes, device, what):
        assert t.numel() == n and t.dtype in dtypes and t.is_contiguous()
        return t.data_ptr()
    monkeypatch.setattr(fff, "_flat", flat)


def tensors(n=300, count=2, bits=8, dtype=B):
    p, g = ([torch.zeros(n, dtype=dtype) for _ in range(count)] for _ in range(2))
    m, v, s = fff.adamw_state(p, bits)
    w = [torch.zeros(n) for _ in range(count)] if dtype is B else None
    return dict(params=p, grads=g, exp_avg=m, exp_avg_sq=v, masters=w, scales=s)


def table(t):
    t = dict(t)
    return fff.adamw_table(t.pop("params"), t.pop("grads"), t.pop("exp_avg"), t.pop("exp_avg_sq"), **t)


@pytest.mark.parametrize("key", ["params", "masters", "exp_avg", "exp_avg_sq", "scales"])
def test_a_tensor_that_two_entries_write_is_refused(on_cpu, key):
    t = tensors()
    assert table(t).count == 2
    t[key][1] = t[key][0]
    with pytest.raises(ValueError, match=rf"{key}\[0\] and {key}\[1\]"):
        table(t)


@pytest.mark.parametrize("key,over", [("params", 1), ("masters", 1), ("exp_avg", 1), ("exp_avg_sq", 299),
                                      ("scales", 2)])
def test_views_that_share_some_elements_are_refused(on_cpu, key, over):
    t = tensors()
    n = t[key][0].numel()
    buf = torch.zeros(2 * n, dtype=torch.uint8 if t[key][0].dtype is F8 else t[key][0].dtype).view(t[key][0].dtype)
    shape = t[key][0].shape
    t[key] = [buf[:n].view(shape), buf[n:].view(shape)]  # side by side
    table(t)
    t[key] = [buf[over:n + over].view(shape), buf[:n].view(shape)]
    with pytest.raises(ValueError, match=rf"{key}\[1\] and {key}\[0\] share memory"):
        table(t)


def test_lists_that_share_a_tensor_are_refused(on_cpu):
    t = tensors(dtype=torch.float32, bits=32)
    t["exp_avg_sq"] = t["exp_avg"]
    with pytest.raises(ValueError, match="exp_avg"):
        table(t)


def test_a_gradient_in_memory_that_another_tensor_writes_is_refused(on_cpu):
    """A lane reads its gradient before it writes its own elements, but other
    workgroups may have written another's."""
    t = tensors(dtype=torch.float32, bits=32)
    t["grads"][1] = t["grads"][0]  # only read: no harm
    table(t)
    t["grads"][0] = t["params"][0]  # element by element its own
    table(t)
    t["grads"][0] = t["params"][1]
    with pytest.raises(ValueError, match=r"grads\[0\] and params\[1\] share memory"):
        table(t)
    buf = torch.zeros(301)
    t["grads"][0], t["params"][0] = buf[:300], buf[1:]
    with pytest.raises(ValueError, match=r"grads\[0\] and params\[0\] share memory"):
        table(t)


def test_empty_tensors_share_nothing(on_cpu):
    t = tensors(dtype=torch.float32, bits=32)
    for key in ("params", "grads", "exp_avg", "exp_avg_sq"):
        t[key].append(t["params"][0][:0])
    assert table(t).count == 3


@pytest.mark.parametrize("key", ["grads", "exp_avg", "exp_avg_sq", "masters", "scales"])
def test_one_tensor_is_not_every_entrys(on_cpu, key):
    t = tensors()
    t[key] = t[key][0]
    with pytest.raises(ValueError, match="one entry for each"):
        table(t)
    one = {k: v[:1] for k, v in tensors().items()}
    one[key] = one[key][0]  # the only entry's
    assert table(one).count == 1


@pytest.mark.parametrize("bits", [8, 32])
def test_a_state_of_parameters_that_can_be_walked_once(on_cpu, bits):
    """Module.parameters() is a generator."""
    module = torch.nn.Linear(30, 20)
    m, v, s = fff.adamw_state(module.parameters(), bits)
    assert [t.shape for t in m] == [t.shape for t in v] == [(20, 30), (20,)]
    assert s is None if bits == 32 else [tuple(t.shape) for t in s] == [(5, 2), (1, 2)]
    grads = (torch.zeros_like(p) for p in module.parameters())
    assert fff.adamw_table(module.parameters(), grads, m, v, scales=s).count == 2


def test_a_captured_norm_has_a_workspace_of_its_own(on_cpu, monkeypatch):
    """Calls on a stream share the table's; a call that is captured gets
    memory of the capture's, which lives as long as the graph, and the table
    holds it besides for captures whose allocations no pool keeps."""
    g = [torch.zeros(300_000)]
    table = fff.grad_table(g)
    assert table.norm_workspace > 0
    used = []

    class Stub:
        def fff_grad_norm(self, entries, count, limit, out, workspace, size, stream):
            used.append(workspace)
            return fff.SUCCESS

    class Capturing:
        now = False

        def __call__(self):
            return self.now

    capturing = Capturing()
    monkeypatch.setattr(fff, "_lib", Stub())
    monkeypatch.setattr(fff, "_here", lambda rt, t, stream: 0)
    monkeypatch.setattr(fff._rt(), "capturing", capturing, raising=False)
    for capturing.now in (False, False, True, True, False):
        fff.grad_norm(table)
    first, second, captured, again, last = used
    assert first == second == last and len({first, captured, again}) == 3
    del captured, again
    held = {w.data_ptr() for w in list(table._workspaces.values()) + table._captured}
    assert held == set(used)


@pytest.mark.parametrize("step", [1 << 63, (1 << 64) + 1, -(1 << 64) + 1])
def test_a_step_beyond_its_field_is_refused(on_cpu, monkeypatch, step):
    """In 64 bits the last two would be the first step."""
    t = table(tensors())
    stub = Library()
    monkeypatch.setattr(fff, "_lib", stub)
    monkeypatch.setattr(fff, "_here", lambda rt, t, stream: 0)
    with pytest.raises(fff.FFFError) as e:
        fff.adamw_step(t, lr=1e-3, step=step)
    assert e.value.status == fff.ERROR_INVALID_VALUE and not stub.shapes
    fff.adamw_step(t, lr=1e-3, step=(1 << 63) - 1)
    assert stub.shapes.pop().step == (1 << 63) - 1
