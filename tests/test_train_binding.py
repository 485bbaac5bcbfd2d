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
