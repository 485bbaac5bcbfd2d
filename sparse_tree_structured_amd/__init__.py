"""Python binding of the FFF forward-pass library (libfff.so, C ABI in
include/fff.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Torch tensors supply device memory and the current stream.  If the
library has not been built this module raises on first use; there is no
fallback implementation.
"""
from __future__ import annotations

import bisect
import ctypes
import functools
import os
from typing import NamedTuple, Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_PKG, "libfff.so")

# fff_dtype_t
DTYPE_F32 = 0
DTYPE_BF16 = 1
DTYPE_E4M3 = 2
# fff_status_t
SUCCESS = 0
ERROR_INVALID_VALUE = 1
ERROR_NOT_SUPPORTED = 2
ERROR_WORKSPACE = 3
ERROR_HIP = 4
# fff_algo_t
ALGO_AUTO = 0
ALGO_GENERIC = 1
ALGO_PREFILL = 2
ALGO_DECODE = 3
ALGOS = {"auto": ALGO_AUTO, "generic": ALGO_GENERIC, "prefill": ALGO_PREFILL, "decode": ALGO_DECODE}
# fff_plan_t flags
PLAN_TEST_DECODE_NO_PUBLISH = 1
# fff_variant_t
VARIANT_FFF = 0
VARIANT_POST = 1
VARIANTS = {"fff": VARIANT_FFF, "post": VARIANT_POST}
# fff_act_t
ACTS = {"none": 0, "gelu": 1, "silu": 2, "relu": 3}
MAX_DEPTH = 20
DENSE_MAX_WIDTH = 1 << 20  # FFF_DENSE_MAX_WIDTH


class Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("P", ctypes.c_int32),
                ("D", ctypes.c_int32), ("h", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("variant", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [("algo", ctypes.c_int32), ("split_level", ctypes.c_int32),
                ("chunk_tokens", ctypes.c_int32), ("flags", ctypes.c_int32)]


class StageEvents(ctypes.Structure):
    """fff_stage_events_t: HIP events recorded at the stage boundaries."""
    _fields_ = [("start", ctypes.c_void_p), ("prepared", ctypes.c_void_p), ("top", ctypes.c_void_p),
                ("deep", ctypes.c_void_p), ("routed", ctypes.c_void_p), ("done", ctypes.c_void_p)]
    NAMES = ("start", "prepared", "top", "deep", "routed", "done")


class Pruning(ctypes.Structure):
    """fff_pruning_t: a prepared static-pruning table (device memory is the
    caller's; keep the tensor that holds it alive while the table is used)."""
    _fields_ = [("table", ctypes.c_void_p), ("P", ctypes.c_int32), ("D", ctypes.c_int32),
                ("d", ctypes.c_int32), ("split_level", ctypes.c_int32),
                ("col_tiles", ctypes.c_int32)]


class NormShape(ctypes.Structure):
    """fff_norm_shape_t."""
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("stream_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("group", ctypes.c_int32), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float)]


class AdamwTensor(ctypes.Structure):
    """fff_adamw_tensor_t."""
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("lr_scale", ctypes.c_double), ("weight_decay", ctypes.c_double)]


class AdamwConfig(ctypes.Structure):
    """fff_adamw_config_t."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64),
                ("state_dtype", ctypes.c_int32), ("stochastic", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("grad_scale", ctypes.c_void_p)]


class DenseShape(ctypes.Structure):
    """fff_dense_shape_t."""
    _fields_ = [("T", ctypes.c_int64), ("K", ctypes.c_int32), ("N", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("save_dtype", ctypes.c_int32), ("save_group", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("x_group", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32)]


class FFFError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


EXPORTS = ("fff_plan_default", "fff_plan_resolve", "fff_workspace_size", "fff_forward",
           "fff_route", "fff_project", "fff_project_workspace_size", "fff_project_ws",
           "fff_status_string", "fff_algo_name",
           "fff_prune_table_size", "fff_prune_prepare", "fff_forward_pruned",
           "fff_backward_workspace_size", "fff_backward", "fff_forward_static",
           "fff_backward_pruned_workspace_size", "fff_backward_pruned",
           "fff_rms_norm", "fff_rms_norm_backward_workspace_size", "fff_rms_norm_backward",
           "fff_adamw_step", "fff_grad_norm_workspace_size", "fff_grad_norm",
           "fff_linear_workspace_size", "fff_linear", "fff_linear_backward_workspace_size",
           "fff_linear_backward", "fff_gated_workspace_size", "fff_gated",
           "fff_gated_backward_workspace_size", "fff_gated_backward",
           "fff_checkpoint_save", "fff_checkpoint_load")
ADAMW_BLOCK = 128  # FFF_ADAMW_BLOCK: elements per scale of an 8-bit state
STATIC_SCRATCH_BYTES = 32 << 20  # FFF_STATIC_SCRATCH_BYTES

_lib: Optional[ctypes.CDLL] = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libfff.so; raises if it is missing (build it with build.py)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIBRARY
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing: build it with `python sparse_tree_structured_amd/build.py` "
                          "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(p)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    SP, PP = ctypes.POINTER(Shape), ctypes.POINTER(Plan)
    lib.fff_plan_default.argtypes = [SP, PP]
    lib.fff_plan_resolve.argtypes = [SP, PP, PP]
    lib.fff_workspace_size.argtypes = [SP, PP, ctypes.POINTER(sz)]
    lib.fff_forward.argtypes = [SP, PP, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                ctypes.POINTER(StageEvents)]
    lib.fff_route.argtypes = [SP, PP, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fff_project.argtypes = [SP, ctypes.c_int32, vp, vp, vp, vp]
    lib.fff_project_workspace_size.argtypes = [SP, ctypes.c_int32, ctypes.POINTER(sz)]
    lib.fff_project_ws.argtypes = [SP, ctypes.c_int32, vp, vp, vp, vp, sz, vp]
    PrP = ctypes.POINTER(Pruning)
    lib.fff_prune_table_size.argtypes = [SP, PP, ctypes.POINTER(sz)]
    lib.fff_prune_prepare.argtypes = [SP, PP, vp, vp, vp, sz, vp, PrP]
    lib.fff_forward_pruned.argtypes = [SP, PP, PrP, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                       ctypes.POINTER(StageEvents)]
    lib.fff_backward_workspace_size.argtypes = [SP, PP, ctypes.POINTER(sz)]
    lib.fff_backward.argtypes = [SP, PP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fff_backward_pruned_workspace_size.argtypes = [SP, PP, PrP, ctypes.POINTER(sz)]
    lib.fff_backward_pruned.argtypes = [SP, PP, PrP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        vp, sz, vp]
    lib.fff_forward_static.argtypes = [SP, PP, vp, vp, vp, vp, vp, vp, vp, vp,
                                       ctypes.POINTER(StageEvents)]
    NP, TP = ctypes.POINTER(NormShape), ctypes.POINTER(AdamwTensor)
    lib.fff_rms_norm.argtypes = [NP, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.fff_rms_norm_backward_workspace_size.argtypes = [NP, ctypes.POINTER(sz)]
    lib.fff_rms_norm_backward.argtypes = [NP, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fff_adamw_step.argtypes = [ctypes.POINTER(AdamwConfig), TP, ctypes.c_int64, vp]
    lib.fff_grad_norm_workspace_size.argtypes = [TP, ctypes.c_int64, ctypes.POINTER(sz)]
    lib.fff_grad_norm.argtypes = [TP, ctypes.c_int64, ctypes.c_double, vp, vp, sz, vp]
    DP, i32, i64 = ctypes.POINTER(DenseShape), ctypes.c_int32, ctypes.c_int64
    for name in ("fff_linear", "fff_gated"):
        getattr(lib, name + "_workspace_size").argtypes = [DP, ctypes.POINTER(sz)]
        getattr(lib, name + "_backward_workspace_size").argtypes = [DP, ctypes.POINTER(sz)]
    lib.fff_linear.argtypes = [DP] + [vp] * 8 + [sz, vp]
    lib.fff_linear_backward.argtypes = [DP] + [vp] * 10 + [sz, vp]
    lib.fff_gated.argtypes = [DP] + [vp] * 9 + [sz, vp]
    lib.fff_gated_backward.argtypes = [DP] + [vp] * 14 + [sz, vp]
    lib.fff_checkpoint_save.argtypes = [i64, i32, i32, i32, vp, vp, vp, vp]
    lib.fff_checkpoint_load.argtypes = [i64, i32, i32, i32, vp, vp, vp, vp]
    lib.fff_status_string.argtypes = [ctypes.c_int]
    lib.fff_status_string.restype = ctypes.c_char_p
    lib.fff_algo_name.argtypes = [ctypes.c_int32]
    lib.fff_algo_name.restype = ctypes.c_char_p
    for name in ("fff_plan_default", "fff_plan_resolve", "fff_workspace_size", "fff_forward",
                 "fff_route", "fff_project", "fff_project_workspace_size", "fff_project_ws",
                 "fff_prune_table_size", "fff_prune_prepare",
                 "fff_forward_pruned", "fff_backward_workspace_size", "fff_backward",
                 "fff_forward_static", "fff_rms_norm", "fff_rms_norm_backward_workspace_size",
                 "fff_rms_norm_backward", "fff_adamw_step", "fff_grad_norm_workspace_size",
                 "fff_grad_norm", "fff_linear_workspace_size", "fff_linear",
                 "fff_linear_backward_workspace_size", "fff_linear_backward",
                 "fff_gated_workspace_size", "fff_gated", "fff_gated_backward_workspace_size",
                 "fff_gated_backward", "fff_checkpoint_save", "fff_checkpoint_load"):
        getattr(lib, name).restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().fff_status_string(int(status)).decode()


def algo_name(algo: int) -> str:
    return load_library().fff_algo_name(int(algo)).decode()


def _variant_code(variant) -> int:
    return VARIANTS[variant] if isinstance(variant, str) else int(variant)


def make_shape(T: int, d: int, P: int, D: int, h: int, dtype: int, variant=VARIANT_FFF) -> Shape:
    return Shape(int(T), int(d), int(P), int(D), int(h), int(dtype), _variant_code(variant))


def make_plan(algo=ALGO_AUTO, split_level: int = -1, chunk_tokens: int = 0,
              flags: int = 0) -> Plan:
    if isinstance(algo, str):
        algo = ALGOS[algo]
    return Plan(int(algo), int(split_level), int(chunk_tokens), int(flags))


def plan_default(shape: Shape) -> Plan:
    p = Plan()
    st = load_library().fff_plan_default(ctypes.byref(shape), ctypes.byref(p))
    if st != SUCCESS:
        raise FFFError(st, "fff_plan_default")
    return p


def resolve_plan(shape: Shape, plan: Plan) -> Plan:
    """The plan as the library would run it ('choose by shape' fields filled in)."""
    out = Plan()
    st = load_library().fff_plan_resolve(ctypes.byref(shape), ctypes.byref(plan), ctypes.byref(out))
    if st != SUCCESS:
        raise FFFError(st, "fff_plan_resolve")
    return out


def workspace_size(shape: Shape, plan: Optional[Plan] = None) -> int:
    n = ctypes.c_size_t()
    st = load_library().fff_workspace_size(ctypes.byref(shape),
                                           ctypes.byref(plan) if plan is not None else None,
                                           ctypes.byref(n))
    if st != SUCCESS:
        raise FFFError(st, "fff_workspace_size")
    return int(n.value)


# ---- torch-facing helpers (device memory and streams only) ----

def _torch():
    import torch
    return torch


def _type_code(dtype, torch) -> int:
    if dtype is torch.float32:
        return DTYPE_F32
    if dtype is torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported dtype {dtype}")


def _dtype_code(t) -> int:
    return _type_code(t.dtype, _torch())


def _dims(t, n, what):
    if t.dim() != n:
        raise ValueError(f"{what} must have {n} dimensions, got shape {tuple(t.shape)}")
    return tuple(int(v) for v in t.shape)


def shape_of(x, W_node, V_node, variant=VARIANT_FFF) -> Shape:
    T, d = _dims(x, 2, "x [T,d]")
    P, N, d2 = _dims(W_node, 3, "W_node [P,N,d]")
    _dims(V_node, 3, "V_node [P,N,h]")
    h = int(V_node.shape[2])
    D = N.bit_length() - 1
    if d2 != d or N < 1 or (1 << (D + 1)) - 1 != N:
        raise ValueError(f"W_node must be [P, 2^(D+1)-1, d={d}], got {tuple(W_node.shape)}")
    return make_shape(T, d, P, D, h, _dtype_code(x), variant)


def _want(t, shape, what):
    if tuple(int(v) for v in t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")


def _check(tensors, dtype, device):
    """Every tensor contiguous, of `dtype`, on `device`, which must be a GPU
    (the library takes device pointers only)."""
    for t in tensors:
        if t.dtype != dtype or t.device != device or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous, on one device, of one dtype")
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, not {device}")


def _check_layer(shape: Shape, x, W_node, b_node, V_node, W_out=None, extra=(), y=None,
                 path_out=None, workspace=None):
    """Full shapes of the layer's tensors against `shape` (W_out in the
    library's [P*h, d] layout, not nn.Linear's [d, P*h]), of the optional
    outputs y [T,d], path_out [T,P] and a flat workspace; then dtype (the
    layer's, int32 for path_out, uint8 for the workspace), device and
    contiguity.  Raises ValueError before anything reaches the library."""
    torch = _torch()
    N = (1 << (shape.D + 1)) - 1
    _want(x, (shape.T, shape.d), "x [T,d]")
    _want(W_node, (shape.P, N, shape.d), "W_node [P,N,d]")
    _want(b_node, (shape.P, N), "b_node [P,N]")
    _want(V_node, (shape.P, N, shape.h), "V_node [P,N,h]")
    same = [x, W_node, b_node, V_node]
    if W_out is not None:
        _want(W_out, (shape.P * shape.h, shape.d), "W_out [P*h,d]")
        same.append(W_out)
    for t, want, what in extra:
        _want(t, want, what)
        same.append(t)
    if y is not None:
        _want(y, (shape.T, shape.d), "y [T,d]")
        same.append(y)
    if path_out is not None:
        _want(path_out, (shape.T, shape.P), "path_out [T,P]")
    if workspace is not None and workspace.dim() != 1:
        raise ValueError("workspace must be a flat uint8 tensor")
    _check(same, x.dtype, x.device)
    if path_out is not None:
        _check([path_out], torch.int32, x.device)
    if workspace is not None:
        _check([workspace], torch.uint8, x.device)


def _stream_handle(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def alloc_workspace(shape: Shape, plan: Optional[Plan], device):
    torch = _torch()
    n = workspace_size(shape, plan)
    # torch's caching allocator returns blocks aligned to at least 512 bytes.
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device), n


def forward(x, W_node, b_node, V_node, W_out, *, algo=ALGO_AUTO, split_level: int = -1,
            chunk_tokens: int = 0, want_path: bool = True, workspace=None, y=None, path_out=None,
            stream=None, events: Optional[StageEvents] = None,
            variant=VARIANT_FFF, plan_flags: int = 0) -> Tuple[object, Optional[object]]:
    """y = FFF(x); returns (y, path_out[T,P] int32 or None).

    ``variant`` "fff" (0) applies GELU to each visited node's logit; "post"
    (1) applies it to each element of a tree's summed output instead.
    ``plan_flags``: fff_plan_t flags (PLAN_TEST_DECODE_NO_PUBLISH, tests only)."""
    torch = _torch()
    shape = shape_of(x, W_node, V_node, variant)
    _check_layer(shape, x, W_node, b_node, V_node, W_out, y=y, path_out=path_out,
                 workspace=workspace)
    plan = make_plan(algo, split_level, chunk_tokens, plan_flags)
    if workspace is None:
        workspace, nbytes = alloc_workspace(shape, plan, x.device)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    if y is None:
        y = torch.empty((shape.T, shape.d), dtype=x.dtype, device=x.device)
    if want_path and path_out is None:
        path_out = torch.empty((shape.T, shape.P), dtype=torch.int32, device=x.device)
    st = load_library().fff_forward(
        ctypes.byref(shape), ctypes.byref(plan), x.data_ptr(), W_node.data_ptr(), b_node.data_ptr(),
        V_node.data_ptr(), W_out.data_ptr(), y.data_ptr(),
        path_out.data_ptr() if path_out is not None else None,
        workspace.data_ptr(), nbytes, _stream_handle(stream),
        ctypes.byref(events) if events is not None else None)
    if st != SUCCESS:
        raise FFFError(st, "fff_forward")
    return y, path_out


def forward_static(x, W_node, b_node, V_node, W_out, y, path_out=None, *, algo=ALGO_AUTO,
                   split_level: int = -1, chunk_tokens: int = 0, stream=None,
                   events: Optional[StageEvents] = None, variant=VARIANT_FFF,
                   plan_flags: int = 0):
    """fff_forward_static: the layer with the library's fixed scratch region
    as its workspace.  The caller passes y [T,d] (and path_out [T,P] int32,
    or None); nothing is allocated."""
    shape = shape_of(x, W_node, V_node, variant)
    _check_layer(shape, x, W_node, b_node, V_node, W_out, y=y, path_out=path_out)
    plan = make_plan(algo, split_level, chunk_tokens, plan_flags)
    st = load_library().fff_forward_static(
        ctypes.byref(shape), ctypes.byref(plan), x.data_ptr(), W_node.data_ptr(),
        b_node.data_ptr(), V_node.data_ptr(), W_out.data_ptr(), y.data_ptr(),
        path_out.data_ptr() if path_out is not None else None, _stream_handle(stream),
        ctypes.byref(events) if events is not None else None)
    if st != SUCCESS:
        raise FFFError(st, "fff_forward_static")
    return y, path_out


def route(x, W_node, b_node, V_node, *, algo=ALGO_AUTO, split_level: int = -1,
          chunk_tokens: int = 0, stream=None, variant=VARIANT_FFF):
    """Routing only: returns (H[T, P*h], path_out[T,P])."""
    torch = _torch()
    shape = shape_of(x, W_node, V_node, variant)
    _check_layer(shape, x, W_node, b_node, V_node)
    plan = make_plan(algo, split_level, chunk_tokens)
    workspace, nbytes = alloc_workspace(shape, plan, x.device)
    H = torch.empty((shape.T, shape.P * shape.h), dtype=x.dtype, device=x.device)
    path = torch.empty((shape.T, shape.P), dtype=torch.int32, device=x.device)
    st = load_library().fff_route(ctypes.byref(shape), ctypes.byref(plan), x.data_ptr(),
                                  W_node.data_ptr(), b_node.data_ptr(), V_node.data_ptr(),
                                  H.data_ptr(), path.data_ptr(), workspace.data_ptr(), nbytes,
                                  _stream_handle(stream))
    if st != SUCCESS:
        raise FFFError(st, "fff_route")
    return H, path


def project_workspace_size(shape: Shape, algo=ALGO_AUTO) -> int:
    """Workspace bytes of fff_project_ws (0 where it needs none)."""
    if isinstance(algo, str):
        algo = ALGOS[algo]
    n = ctypes.c_size_t()
    st = load_library().fff_project_workspace_size(ctypes.byref(shape), int(algo), ctypes.byref(n))
    if st != SUCCESS:
        raise FFFError(st, "fff_project_workspace_size")
    return n.value


def project(H, W_out, *, algo=ALGO_AUTO, stream=None, y=None, workspace=None,
            use_workspace: bool = True):
    """y = H . W_out (fp32 accumulation).

    With ``use_workspace`` (default) the call goes through fff_project_ws
    (whose workspace size is 0: it may be None), else through fff_project;
    both run the kernel fff_forward's projection uses for the same shape."""
    torch = _torch()
    T, K = _dims(H, 2, "H [T,K]")
    K2, d = _dims(W_out, 2, "W_out [K,d]")
    if K2 != K:
        raise ValueError(f"H {list(H.shape)} and W_out {list(W_out.shape)} disagree on K")
    if y is not None:
        _want(y, (T, d), "y [T,d]")
    _check([H, W_out] + ([y] if y is not None else []), H.dtype, H.device)
    if workspace is not None:
        _check([workspace], torch.uint8, H.device)
    # K = P*h with P=1, h=K describes the product for the library.
    shape = make_shape(T, d, 1, 0, K, _dtype_code(H))
    if y is None:
        y = torch.empty((T, d), dtype=H.dtype, device=H.device)
    if isinstance(algo, str):
        algo = ALGOS[algo]
    lib = load_library()
    if not use_workspace:
        st = lib.fff_project(ctypes.byref(shape), int(algo), H.data_ptr(), W_out.data_ptr(),
                             y.data_ptr(), _stream_handle(stream))
        if st != SUCCESS:
            raise FFFError(st, "fff_project")
        return y
    if workspace is None:
        nbytes = project_workspace_size(shape, algo)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=H.device) if nbytes else None
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.fff_project_ws(ctypes.byref(shape), int(algo), H.data_ptr(), W_out.data_ptr(),
                            y.data_ptr(), ws_ptr, ws_bytes, _stream_handle(stream))
    if st != SUCCESS:
        raise FFFError(st, "fff_project_ws")
    return y


def prune_table_size(shape: Shape, plan: Optional[Plan] = None) -> int:
    n = ctypes.c_size_t()
    st = load_library().fff_prune_table_size(ctypes.byref(shape),
                                             ctypes.byref(plan) if plan is not None else None,
                                             ctypes.byref(n))
    if st != SUCCESS:
        raise FFFError(st, "fff_prune_table_size")
    return int(n.value)


def prune_prepare(leaf_alive, W_node, V_node, *, algo=ALGO_AUTO, split_level: int = -1,
                  chunk_tokens: int = 0, T: Optional[int] = None, stream=None,
                  variant=VARIANT_FFF):
    """Static path pruning table for trees W_node [P,N,d] (device) and a leaf
    mask leaf_alive [P, 2^D] (host: numpy or CPU tensor, nonzero = alive).
    The plan is resolved for T tokens (default 65536, a prefill batch) and
    the given options; returns (Pruning, table tensor), the tensor owning the
    device memory."""
    import numpy as np
    torch = _torch()
    P, N, d = W_node.shape
    D = N.bit_length() - 1
    mask = np.ascontiguousarray(np.asarray(leaf_alive, dtype=np.uint8))
    if mask.shape != (P, 1 << D):
        raise ValueError("leaf_alive must be [P, 2^D]")
    shape = make_shape(T if T is not None else 65536, d, P, D, V_node.shape[2],
                       _dtype_code(W_node), variant)
    plan = make_plan(algo, split_level, chunk_tokens)
    n = prune_table_size(shape, plan)
    table = torch.empty(max(n, 1), dtype=torch.uint8, device=W_node.device)
    out = Pruning()
    st = load_library().fff_prune_prepare(
        ctypes.byref(shape), ctypes.byref(plan), mask.ctypes.data_as(ctypes.c_void_p),
        W_node.data_ptr(), table.data_ptr(), n, _stream_handle(stream), ctypes.byref(out))
    if st != SUCCESS:
        raise FFFError(st, "fff_prune_prepare")
    return out, table


def forward_pruned(x, W_node, b_node, V_node, W_out, pruning: Pruning, *, algo=ALGO_AUTO,
                   split_level: int = -1, chunk_tokens: int = 0, want_path: bool = True,
                   workspace=None, y=None, path_out=None, stream=None,
                   events: Optional[StageEvents] = None, variant=VARIANT_FFF):
    """fff_forward_pruned: y and path_out of the pruned trees."""
    torch = _torch()
    shape = shape_of(x, W_node, V_node, variant)
    _check_layer(shape, x, W_node, b_node, V_node, W_out, y=y, path_out=path_out,
                 workspace=workspace)
    plan = make_plan(algo, split_level, chunk_tokens)
    if workspace is None:
        workspace, nbytes = alloc_workspace(shape, plan, x.device)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    if y is None:
        y = torch.empty((shape.T, shape.d), dtype=x.dtype, device=x.device)
    if want_path and path_out is None:
        path_out = torch.empty((shape.T, shape.P), dtype=torch.int32, device=x.device)
    st = load_library().fff_forward_pruned(
        ctypes.byref(shape), ctypes.byref(plan), ctypes.byref(pruning), x.data_ptr(),
        W_node.data_ptr(), b_node.data_ptr(), V_node.data_ptr(), W_out.data_ptr(), y.data_ptr(),
        path_out.data_ptr() if path_out is not None else None, workspace.data_ptr(), nbytes,
        _stream_handle(stream), ctypes.byref(events) if events is not None else None)
    if st != SUCCESS:
        raise FFFError(st, "fff_forward_pruned")
    return y, path_out


def backward_workspace_size(shape: Shape, plan: Optional[Plan] = None) -> int:
    n = ctypes.c_size_t()
    st = load_library().fff_backward_workspace_size(
        ctypes.byref(shape), ctypes.byref(plan) if plan is not None else None, ctypes.byref(n))
    if st != SUCCESS:
        raise FFFError(st, "fff_backward_workspace_size")
    return int(n.value)


def backward_pruned_workspace_size(shape: Shape, plan: Optional[Plan], pruning: Pruning) -> int:
    n = ctypes.c_size_t()
    st = load_library().fff_backward_pruned_workspace_size(
        ctypes.byref(shape), ctypes.byref(plan) if plan is not None else None,
        ctypes.byref(pruning), ctypes.byref(n))
    if st != SUCCESS:
        raise FFFError(st, "fff_backward_pruned_workspace_size")
    return int(n.value)


def backward(x, W_node, b_node, V_node, W_out, dy, *, algo=ALGO_AUTO, split_level: int = -1,
             workspace=None, out=None, stream=None, variant=VARIANT_FFF):
    """Gradients of sum(y * dy) with the forward's paths held fixed.  Returns
    a dict: dx (dtype of x), dW_node, db_node, dV_node, dW_out (float32)."""
    return _backward(x, W_node, b_node, V_node, W_out, dy, None, algo, split_level, workspace,
                     out, stream, variant)


def backward_pruned(x, W_node, b_node, V_node, W_out, dy, pruning: Pruning, *, algo=ALGO_AUTO,
                    split_level: int = -1, workspace=None, out=None, stream=None,
                    variant=VARIANT_FFF):
    """fff_backward_pruned: the gradients of backward() with the paths
    fff_forward_pruned takes on the prepared table."""
    return _backward(x, W_node, b_node, V_node, W_out, dy, pruning, algo, split_level, workspace,
                     out, stream, variant)


def _backward(x, W_node, b_node, V_node, W_out, dy, pruning, algo, split_level, workspace, out,
              stream, variant):
    torch = _torch()
    shape = shape_of(x, W_node, V_node, variant)
    N = (1 << (shape.D + 1)) - 1
    want = {"dx": ((shape.T, shape.d), x.dtype), "dW_node": ((shape.P, N, shape.d), torch.float32),
            "db_node": ((shape.P, N), torch.float32),
            "dV_node": ((shape.P, N, shape.h), torch.float32),
            "dW_out": ((shape.P * shape.h, shape.d), torch.float32)}
    if out is not None:
        for k, (shp, _) in want.items():
            _want(out[k], shp, k)
    _check_layer(shape, x, W_node, b_node, V_node, W_out,
                 extra=[(dy, (shape.T, shape.d), "dy [T,d]")], workspace=workspace)
    if out is not None:
        for k, (_, dt) in want.items():
            _check([out[k]], dt, x.device)
    plan = make_plan(algo, split_level, 0)
    if workspace is None:
        n = (backward_workspace_size(shape, plan) if pruning is None
             else backward_pruned_workspace_size(shape, plan, pruning))
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=x.device)
    nbytes = workspace.numel() * workspace.element_size()
    f32 = dict(dtype=torch.float32, device=x.device)
    g = out or {"dx": torch.empty_like(x), "dW_node": torch.empty(W_node.shape, **f32),
                "db_node": torch.empty(b_node.shape, **f32),
                "dV_node": torch.empty(V_node.shape, **f32),
                "dW_out": torch.empty(W_out.shape, **f32)}
    ptrs = (x.data_ptr(), W_node.data_ptr(), b_node.data_ptr(), V_node.data_ptr(),
            W_out.data_ptr(), dy.data_ptr(), g["dx"].data_ptr(), g["dW_node"].data_ptr(),
            g["db_node"].data_ptr(), g["dV_node"].data_ptr(), g["dW_out"].data_ptr(),
            workspace.data_ptr(), nbytes, _stream_handle(stream))
    lib = load_library()
    if pruning is None:
        st = lib.fff_backward(ctypes.byref(shape), ctypes.byref(plan), *ptrs)
        what = "fff_backward"
    else:
        st = lib.fff_backward_pruned(ctypes.byref(shape), ctypes.byref(plan),
                                     ctypes.byref(pruning), *ptrs)
        what = "fff_backward_pruned"
    if st != SUCCESS:
        raise FFFError(st, what)
    return g


# ---- around the layer: norm and optimiser ----

class RmsNorm(NamedTuple):
    """rms_norm's outputs; None where not asked for or not there."""
    y: object             # [T,d], the layer's dtype or float8_e4m3fn
    residual_out: object  # [T,d] x + residual
    rstd: object          # [T] float32, for the backward pass
    scale: object         # [T, groups] float32 beside an 8-bit y


class RmsNormGrad(NamedTuple):
    dz: object       # [T,d] of the residual stream's dtype: the gradient of x and of the residual
    dx: object       # [T,d] the same in the layer's dtype (dz itself where the dtypes agree)
    dweight: object  # [d] float32


@functools.lru_cache(maxsize=256)
def _norm_shape(T, d, dtype, stream_dtype, out_dtype, group, eps, weight_offset) -> NormShape:
    """The descriptor of these sizes, which the library only reads: one for
    each set of values.  ctypes cuts a number that its field cannot hold, and
    the library would see another size than the tensors have."""
    s = NormShape(T, d, dtype, stream_dtype, out_dtype, group, eps, weight_offset)
    if s.d != d:
        raise FFFError(ERROR_NOT_SUPPORTED, f"norm of rows of {d} columns")
    if s.group != group:
        raise FFFError(ERROR_INVALID_VALUE, f"norm with group {group}")
    return s


class _Torch:
    """What a call needs of torch, looked up once: small calls are bound by
    the host."""

    def __init__(self):
        import torch
        self.f32, self.bf16, self.f8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
        self.u8 = torch.uint8
        self.codes = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
        self.empty, self.stream = torch.empty, torch.cuda.stream
        self.device = getattr(torch._C, "_cuda_getDevice", None)
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)


_lazy: Optional[_Torch] = None


def _rt() -> _Torch:
    global _lazy
    if _lazy is None:
        _lazy = _Torch()
    return _lazy


def _here(rt, t, stream):
    """The handle of the stream to launch on: `stream`, or the current one.
    The library launches on the current device, so tensors must be there."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"tensors must be on a GPU, not {t.device}")
    if index != rt.device():
        raise ValueError(f"tensors are on {t.device}, which is not the current device")
    return rt.raw_stream(index) if stream is None else int(stream.cuda_stream)


def _empty(rt, shape, dtype, device, stream):
    """A new tensor that belongs to the stream it is used on."""
    if stream is None:
        return rt.empty(shape, dtype=dtype, device=device)
    with rt.stream(stream):
        return rt.empty(shape, dtype=dtype, device=device)


def _capturing(rt, stream) -> bool:
    if stream is None:
        return rt.capturing()
    with rt.stream(stream):
        return rt.capturing()


def _code(rt, dtype) -> int:
    code = rt.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _tensor(t, shape, dtype, like, what):
    """The pointer of a tensor that must have this shape and dtype, be
    contiguous, and lie on the device of `like`."""
    if (t.shape == shape and t.dtype is dtype and t.is_contiguous()
            and t.get_device() == like.get_device()):
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if t.device != like.device:
        raise ValueError(f"{what} must be on {like.device}, got {t.device}")
    raise ValueError(f"{what} must be contiguous")


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, weight_offset: float = 0.0,
             out_dtype=None, group: int = 0, y=None, scale=None, residual_out=None, rstd=None,
             want_rstd: bool = False, stream=None) -> RmsNorm:
    """fff_rms_norm: y = z * rstd * (weight + weight_offset) with
    z = x + residual, over rows [T,d].

    The layer's dtype is the weight's, else x's; the residual (and
    residual_out) may be float32 beside a bf16 layer, and so may x where
    there is no residual.  ``out_dtype`` torch.float8_e4m3fn (or a ``y`` of
    that dtype) gives y in 8 bits with a scale per row, or per ``group`` = 32,
    64 or 128 columns.  ``residual_out`` may be ``residual`` itself."""
    rt = _rt()
    shape, ty = x.shape, x.dtype
    if len(shape) != 2:
        raise ValueError(f"x [T,d] must have 2 dimensions, got shape {tuple(shape)}")
    T, d = shape
    stream_ty = ty if residual is None else residual.dtype
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    px, pr, pw, pz, prs, ps = x.data_ptr(), 0, 0, 0, 0, 0
    if weight is not None:
        ty = weight.dtype
        pw = _tensor(weight, (d,), ty, x, "weight [d]")
    if residual is not None:
        pr = _tensor(residual, shape, stream_ty, x, "residual")
        if x.dtype is not ty:
            raise ValueError(f"x must be {ty} beside a residual, got {x.dtype}")
    code, stream_code = _code(rt, ty), _code(rt, stream_ty)
    out_ty = y.dtype if y is not None else (out_dtype or ty)
    if out_dtype is not None and out_ty is not out_dtype:
        raise ValueError(f"y must be {out_dtype}, got {out_ty}")
    e4m3 = out_ty is rt.f8
    if not e4m3 and out_ty is not ty:
        raise ValueError(f"y must be {ty} or {rt.f8}, got {out_ty}")
    sizes = _norm_shape(T, d, code, stream_code, DTYPE_E4M3 if e4m3 else code, group, eps, weight_offset)
    handle = _here(rt, x, stream)
    if residual is None and stream_ty is not ty:  # x is the stream itself
        px, pr = 0, px
    if y is not None:
        py = _tensor(y, shape, out_ty, x, "y")
    else:
        y = _empty(rt, shape, out_ty, x.device, stream)
        py = y.data_ptr()
    if residual_out is not None:
        pz = _tensor(residual_out, shape, stream_ty, x, "residual_out")
    elif residual is not None:
        residual_out = _empty(rt, shape, stream_ty, x.device, stream)
        pz = residual_out.data_ptr()
    if rstd is not None:
        prs = _tensor(rstd, (T,), rt.f32, x, "rstd [T]")
    elif want_rstd:
        rstd = _empty(rt, (T,), rt.f32, x.device, stream)
        prs = rstd.data_ptr()
    if e4m3:
        groups = (T, -(-d // group) if group > 0 else 1)
        if scale is not None:
            ps = _tensor(scale, groups, rt.f32, x, "scale [T, groups]")
        else:
            scale = _empty(rt, groups, rt.f32, x.device, stream)
            ps = scale.data_ptr()
    elif scale is not None:
        raise ValueError(f"scale is for a y of {rt.f8}")
    st = (_lib or load_library()).fff_rms_norm(sizes, px, pr, pw, py, ps, pz, prs, handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_rms_norm")
    return RmsNorm(y, residual_out, rstd, scale)


@functools.lru_cache(maxsize=256)
def rms_norm_backward_workspace_size(T: int, d: int, dtype: int, stream_dtype: int) -> int:
    """Workspace bytes of rms_norm_backward (dtypes: fff_dtype_t codes)."""
    n = ctypes.c_size_t()
    st = load_library().fff_rms_norm_backward_workspace_size(
        _norm_shape(T, d, dtype, stream_dtype, dtype, 0, 0.0, 0.0), ctypes.byref(n))
    if st != SUCCESS:
        raise FFFError(st, "fff_rms_norm_backward_workspace_size")
    return n.value


def rms_norm_backward(dy, z, weight, rstd, *, dresidual=None, weight_offset: float = 0.0, dz=None,
                      dx=None, dweight=None, want_dweight: bool = True, workspace=None,
                      stream=None) -> RmsNormGrad:
    """fff_rms_norm_backward: the gradients of rms_norm's inputs.  ``z`` is
    what it normalised (its residual_out, or x), ``rstd`` its rstd and
    ``dresidual`` the gradient that reaches residual_out.  Where z is float32
    beside a bf16 layer, dx is dz once more in bf16."""
    rt = _rt()
    shape, ty, zty, f32 = dy.shape, dy.dtype, z.dtype, rt.f32
    if len(shape) != 2:
        raise ValueError(f"dy [T,d] must have 2 dimensions, got shape {tuple(shape)}")
    T, d = shape
    if not dy.is_contiguous():
        raise ValueError("dy must be contiguous")
    pdy = dy.data_ptr()
    pz = _tensor(z, shape, zty, dy, "z")
    pw = _tensor(weight, (d,), ty, dy, "weight [d]") if weight is not None else 0
    pr = _tensor(rstd, (T,), f32, dy, "rstd [T]")
    pe = _tensor(dresidual, shape, zty, dy, "dresidual") if dresidual is not None else 0
    code, zcode = _code(rt, ty), _code(rt, zty)
    sizes = _norm_shape(T, d, code, zcode, code, 0, 0.0, weight_offset)
    handle = _here(rt, dy, stream)
    pdx = pdw = pws = have = 0
    if dz is not None:
        pdz = _tensor(dz, shape, zty, dy, "dz")
    else:
        dz = _empty(rt, shape, zty, dy.device, stream)
        pdz = dz.data_ptr()
    if dx is not None:
        pdx = _tensor(dx, shape, ty, dy, "dx")
    elif zty is not ty:
        dx = _empty(rt, shape, ty, dy.device, stream)
        pdx = dx.data_ptr()
    if dweight is not None:
        pdw = _tensor(dweight, (d,), f32, dy, "dweight [d]")
    elif want_dweight:
        dweight = _empty(rt, (d,), f32, dy.device, stream)
        pdw = dweight.data_ptr()
    if workspace is not None:
        have = workspace.numel()
        pws = _tensor(workspace, (have,), rt.u8, dy, "workspace")
    elif dweight is not None:
        have = rms_norm_backward_workspace_size(T, d, code, zcode)
        if have:
            workspace = _empty(rt, (have,), rt.u8, dy.device, stream)
            pws = workspace.data_ptr()
    st = (_lib or load_library()).fff_rms_norm_backward(
        sizes, pdy, pz, pw, pr, pe, pdz, pdx, pdw, pws, have, handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_rms_norm_backward")
    return RmsNormGrad(dz, dz if dx is None else dx, dweight)


class TensorTable:
    """The tensors of an optimiser, laid out for the library: made once by
    adamw_table or grad_table, used at every step.  It holds their addresses
    and keeps the tensors alive; they are updated in place.  Where a tensor is
    replaced, make another table: after zero_grad(set_to_none=True) the next
    backward pass leaves other gradients in p.grad, and a step on this table
    would read the old ones (zero them in place, or let the backward write
    into them).  One stream uses it at a time, as for the tensors themselves.
    A captured graph holds the tensors' addresses too and does not keep them
    alive: keep the tensors, or the table, as long as the graph."""

    def __init__(self, entries, first, state_code, keep):
        self.entries = entries        # array of AdamwTensor
        self.count = len(entries)
        self.first = first            # the first tensor, for its device
        self.device = first.device
        self.state_code = state_code  # None: gradients only
        self.keep = keep
        n = ctypes.c_size_t()
        st = load_library().fff_grad_norm_workspace_size(entries, self.count, ctypes.byref(n))
        if st != SUCCESS:
            raise FFFError(st, "fff_grad_norm_workspace_size")
        self.norm_workspace = n.value
        self._workspaces = {}  # grad_norm's workspace on every stream that has used the table
        self._captured = []    # and those of its captured calls


def _flat(t, n, dtypes, device, what):
    """The pointer of a contiguous tensor of n elements of one of `dtypes`."""
    if t.numel() != n:
        raise ValueError(f"{what} must have {n} elements, got {list(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous and on {device}")
    if device.type != "cuda":
        raise ValueError(f"{what} must be on a GPU, not {device}")
    return t.data_ptr()


def _listed(values, n, what):
    values = list(values) if isinstance(values, (list, tuple)) else [values] * n
    if len(values) != n:
        raise ValueError(f"{what} must have one entry for each of {n} tensors, got {len(values)}")
    return values


def _tensors(values, n, what, torch):
    """A list of n tensors; None is n of them."""
    if values is None:
        return [None] * n
    # A tensor would list its rows; two entries must not share one.
    values = [values] if isinstance(values, torch.Tensor) else list(values)
    if len(values) != n:
        raise ValueError(f"{what} must have one entry for each of {n} tensors, got {len(values)}")
    return values


def grad_table(grads) -> TensorTable:
    """A table of gradients alone, for grad_norm."""
    torch = _torch()
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    entries = (AdamwTensor * len(grads))()
    for i, (e, g) in enumerate(zip(entries, grads)):
        e.grad = _flat(g, g.numel(), (torch.float32, torch.bfloat16), grads[0].device, f"grads[{i}]")
        e.n, e.grad_dtype = g.numel(), _dtype_code(g)
    return TensorTable(entries, grads[0], None, grads)


def _check_apart(written, grads):
    """Refuses a table whose step would write some memory twice, or read a
    gradient where it writes: workgroups run in any order.  A gradient may be
    a buffer of its own entry, whose elements a lane reads before it writes.
    ``written``: (start, end, entry, name) of what is; ``grads``: (start, end,
    entry)."""
    written.sort()
    for before, w in zip(written, written[1:]):
        if w[0] < before[1]:
            (_, _, i, a), (_, _, j, b) = before, w
            raise ValueError(f"{a}[{i}] and {b}[{j}] share memory: every param, master, state and scale "
                             "must be its own")
    starts = [w[0] for w in written]
    for start, end, i in grads:
        # the last written one that starts before the gradient ends: none before it reaches further
        k = bisect.bisect_left(starts, end) - 1
        if k >= 0 and written[k][1] > start and written[k][:3] != (start, end, i):
            raise ValueError(f"grads[{i}] and {written[k][3]}[{written[k][2]}] share memory")


def adamw_state(params, bits: int = 32):
    """The state before the first step, as adamw_table takes it: lists
    (exp_avg, exp_avg_sq, scales), float32, or for ``bits`` = 8 float8_e4m3fn
    with scales [blocks, 2] (else None)."""
    torch = _torch()
    params = list(params)
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    if bits == 32:
        make = lambda p: torch.zeros(p.shape, dtype=torch.float32, device=p.device)  # noqa: E731
        return [make(p) for p in params], [make(p) for p in params], None
    make = lambda p: torch.zeros(p.shape, dtype=torch.uint8,  # noqa: E731
                                 device=p.device).view(torch.float8_e4m3fn)
    scales = [torch.zeros(-(-p.numel() // ADAMW_BLOCK), 2, dtype=torch.float32, device=p.device)
              for p in params]
    return [make(p) for p in params], [make(p) for p in params], scales


def adamw_table(params, grads, exp_avg, exp_avg_sq, *, masters=None, scales=None,
                weight_decay=0.0, lr_scale=1.0) -> TensorTable:
    """The tensors of an AdamW step: float32 or bf16 params and grads, states
    of one dtype (float32, or float8_e4m3fn with ``scales``; adamw_state makes
    them).  ``masters``: float32 masters of bf16 params (None, or a list with
    None where a param has none).  ``weight_decay`` and ``lr_scale``: one
    number, or one for each tensor.  No two tensors that a step writes may
    share memory."""
    torch, rt = _torch(), _rt()
    params = list(params)
    n = len(params)
    if n == 0:
        raise ValueError("params must hold at least one tensor")
    dev = params[0].device
    f32, both = (torch.float32,), (torch.float32, torch.bfloat16)
    lists = {"grads": grads, "exp_avg": exp_avg, "exp_avg_sq": exp_avg_sq,
             "masters": masters, "scales": scales}  # in the order of the loop below
    lists = {k: _tensors(v, n, k, torch) for k, v in lists.items()}
    decays, shares = _listed(weight_decay, n, "weight_decay"), _listed(lr_scale, n, "lr_scale")
    state = (lists["exp_avg"][0].dtype,)
    e4m3 = state[0] == torch.float8_e4m3fn
    if not e4m3 and state != f32:
        raise ValueError(f"exp_avg must be torch.float32 or torch.float8_e4m3fn, got {state[0]}")
    entries = (AdamwTensor * n)()
    written, read, size = [], [], 1 if e4m3 else 4
    for i, (e, p, g, m, v, w, sc) in enumerate(zip(entries, params, *lists.values())):
        e.n = k = p.numel()
        e.param = pp = _flat(p, k, both, dev, f"params[{i}]")
        e.grad = pg = _flat(g, k, both, dev, f"grads[{i}]")
        e.exp_avg = pm = _flat(m, k, state, dev, f"exp_avg[{i}]")
        e.exp_avg_sq = pv = _flat(v, k, state, dev, f"exp_avg_sq[{i}]")
        e.param_dtype, e.grad_dtype = code, grad_code = rt.codes[p.dtype], rt.codes[g.dtype]
        if k:
            written += ((pp, pp + (2 if code == DTYPE_BF16 else 4) * k, i, "params"),
                        (pm, pm + size * k, i, "exp_avg"), (pv, pv + size * k, i, "exp_avg_sq"))
            read.append((pg, pg + (2 if grad_code == DTYPE_BF16 else 4) * k, i))
        if w is not None:
            if p.dtype != torch.bfloat16:
                raise ValueError(f"masters[{i}] is for a bf16 param, params[{i}] is {p.dtype}")
            e.master = pw = _flat(w, k, f32, dev, f"masters[{i}]")
            if k:
                written.append((pw, pw + 4 * k, i, "masters"))
        if e4m3 != (sc is not None):
            raise ValueError("scales go with exp_avg of torch.float8_e4m3fn, and only with it")
        if e4m3:
            blocks = -(-k // ADAMW_BLOCK)
            e.scale = ps = _flat(sc, 2 * blocks, f32, dev, f"scales[{i}]")
            if k:
                written.append((ps, ps + 8 * blocks, i, "scales"))
        e.lr_scale, e.weight_decay = float(shares[i]), float(decays[i])
    _check_apart(written, read)
    return TensorTable(entries, params[0], DTYPE_E4M3 if e4m3 else DTYPE_F32, (params, lists))


def adamw_step(table: TensorTable, *, lr: float, step: int, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, grad_scale=None, seed: Optional[int] = None,
               stream=None) -> None:
    """fff_adamw_step on a table's tensors, in place.  ``step`` counts from 1.
    ``grad_scale``: a float32 device tensor of one element that multiplies
    every gradient (grad_norm's second value), or None; if it holds NaN the
    step changes nothing.  ``seed``: None rounds to nearest, a number (another
    one at every step) rounds 8-bit states and bf16 params without a master
    stochastically."""
    rt = _rt()
    if table.state_code is None:
        raise ValueError("the table holds gradients only: make it with adamw_table")
    ps = 0
    if grad_scale is not None:
        ps = _flat(grad_scale, 1, (rt.f32,), table.device, "grad_scale")
    handle = _here(rt, table.first, stream)
    config = AdamwConfig(lr, beta1, beta2, eps, step, table.state_code, seed is not None,
                         0 if seed is None else seed & 0xFFFFFFFFFFFFFFFF, ps)
    if config.step != step:  # cut to its field
        raise FFFError(ERROR_INVALID_VALUE, f"AdamW step {step}")
    st = (_lib or load_library()).fff_adamw_step(config, table.entries, table.count, handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_adamw_step")


def grad_norm(grads, *, max_norm: float = float("inf"), out=None, workspace=None, stream=None):
    """fff_grad_norm of a TensorTable or a list of tensors: a float32 device
    tensor [2], the norm of all gradients together and the factor
    min(1, max_norm / (norm + 1e-6)) (NaN where the norm is not finite) that
    adamw_step takes as ``grad_scale`` (``out[1:]``)."""
    rt = _rt()
    table = grads if isinstance(grads, TensorTable) else grad_table(grads)
    handle = _here(rt, table.first, stream)
    pws = have = 0
    if out is None:
        out = _empty(rt, (2,), rt.f32, table.device, stream)
        pout = out.data_ptr()
    else:
        pout = _tensor(out, (2,), rt.f32, table.first, "out [2]")
    if workspace is not None:
        have = workspace.numel()
        pws = _tensor(workspace, (have,), rt.u8, table.first, "workspace")
    elif table.norm_workspace:
        have = table.norm_workspace
        if _capturing(rt, stream):
            # From the capture's own memory, which the graph keeps: the table may
            # go first, and a call beside a replay does not share it.
            workspace = _empty(rt, (have,), rt.u8, table.device, stream)
            table._captured.append(workspace)
        else:
            workspace = table._workspaces.get(handle)
            if workspace is None:
                workspace = table._workspaces[handle] = _empty(rt, (have,), rt.u8, table.device, stream)
        pws = workspace.data_ptr()
    st = (_lib or load_library()).fff_grad_norm(table.entries, table.count, max_norm, pout, pws, have, handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_grad_norm")
    return out


# ---- dense feed-forward block ----

class Checkpoint(NamedTuple):
    """Rows kept in 8 bits: what checkpoint() makes, linear() and gated() save
    and their backward passes read.  rms_norm's 8-bit output is one too:
    Checkpoint(o.y, o.scale, group)."""
    codes: object  # [T,d] float8_e4m3fn
    scale: object  # [T, groups] float32 ([T, 1] with group 0)
    group: int     # columns per scale, 0: the row


class Linear(NamedTuple):
    y: object    # [T,N]
    pre: object  # [T,N] before the activation: a tensor, a Checkpoint, or None


class LinearGrad(NamedTuple):
    dx: object     # [T,K], or None where not asked for (so the others)
    dW: object     # [K,N]
    dbias: object  # [N] float32


class Gated(NamedTuple):
    h: object     # [T,F] act(x . W_gate) * (x . W_up)
    gate: object  # [T,F] x . W_gate: a tensor, a Checkpoint, or None
    up: object    # [T,F] x . W_up


class GatedGrad(NamedTuple):
    dx: object      # [T,d], or None where not asked for (so the others)
    dW_gate: object  # [d,F]
    dW_up: object   # [d,F]
    h: object       # [T,F] made again from gate and up


@functools.lru_cache(maxsize=256)
def _dense(name, T, K, N, dtype, out_dtype, act, save_dtype, save_group, x_dtype, x_group,
           grad_dtype):
    """The descriptor of these sizes, which the library only reads, and the
    workspace bytes of the entry point `name` on them."""
    s = DenseShape(T, K, N, dtype, out_dtype, act, save_dtype, save_group, x_dtype, x_group,
                   grad_dtype)
    # ctypes cuts a number that its field cannot hold
    if s.K != K or s.N != N:
        raise FFFError(ERROR_NOT_SUPPORTED, f"{name} of {K} inputs and {N} outputs")
    if s.save_group != save_group or s.x_group != x_group:
        raise FFFError(ERROR_INVALID_VALUE, f"{name} with groups {save_group}, {x_group}")
    n = ctypes.c_size_t()
    st = getattr(load_library(), name + "_workspace_size")(ctypes.byref(s), ctypes.byref(n))
    if st != SUCCESS:
        raise FFFError(st, name)
    return s, n.value


def _act_code(act) -> int:
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, got {act!r}")
    return code


def _matrix(t, what):
    """The shape of a contiguous matrix."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must have 2 dimensions, got shape {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return shape


def _columns(t, what):
    """Columns of what _tensor then checks as a whole."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must have 2 dimensions, got shape {tuple(shape)}")
    return shape[1]


def _scales(T, d, group):
    return (T, -(-d // group) if group > 0 else 1)


def _kept(rt, t, shape, ty, like, what):
    """Pointers, dtype code and group of a tensor or a Checkpoint."""
    if isinstance(t, Checkpoint):
        if not isinstance(t.group, int) or t.group not in (0, 32, 64, 128):
            raise ValueError(f"{what} must have group 0, 32, 64 or 128, got {t.group}")
        scale = _tensor(t.scale, _scales(*shape, t.group), rt.f32, like, f"{what}'s scale")
        return _tensor(t.codes, shape, rt.f8, like, f"{what}'s codes"), scale, DTYPE_E4M3, t.group
    return _tensor(t, shape, ty, like, what), 0, _code(rt, ty), 0


def _workspace(rt, workspace, need, like, stream):
    """A workspace tensor, its pointer and its bytes."""
    if workspace is not None:
        have = workspace.numel()
        return workspace, _tensor(workspace, (have,), rt.u8, like, "workspace"), have
    if not need:
        return None, 0, 0
    # (an int for the size: a tuple takes longer)
    workspace = rt.empty(need, dtype=rt.u8, device=like.device) if stream is None else \
        _empty(rt, (need,), rt.u8, like.device, stream)
    return workspace, workspace.data_ptr(), need


def _output(rt, t, shape, dtype, like, what, stream):
    """An output tensor, made where there is none, and its pointer."""
    if t is not None:
        return t, _tensor(t, shape, dtype, like, what)
    t = rt.empty(shape, dtype=dtype, device=like.device) if stream is None else \
        _empty(rt, shape, dtype, like.device, stream)
    return t, t.data_ptr()


def _save_kind(rt, save, group, ty, code):
    """Dtype code and group of what is saved."""
    if save not in ("same", "e4m3"):
        raise ValueError(f'save must be None, "same" or "e4m3", got {save!r}')
    return (DTYPE_E4M3, group) if save == "e4m3" else (code, 0)


def _saved(rt, save, group, shape, ty, like, stream):
    """A tensor or Checkpoint for saved sums, and its pointers."""
    t = _empty(rt, shape, rt.f8 if save == "e4m3" else ty, like.device, stream)
    if save == "same":
        return t, t.data_ptr(), 0
    scale = _empty(rt, _scales(*shape, group), rt.f32, like.device, stream)
    return Checkpoint(t, scale, group), t.data_ptr(), scale.data_ptr()


def linear(x, W, bias=None, *, residual=None, act: str = "none", out_dtype=None,
           save: Optional[str] = None, group: int = 128, y=None, workspace=None,
           stream=None) -> Linear:
    """fff_linear: y = act(x . W + bias) + residual, x [T,K], W [K,N].

    ``act``: "none", "gelu" (tanh form), "silu" or "relu".  y and the residual
    are of the layer's dtype, or float32 beside a bf16 layer (``out_dtype``,
    else the residual's or y's dtype); ``y`` may be ``residual`` itself.
    ``save`` keeps x . W + bias for linear_backward: "same" in the layer's
    dtype, "e4m3" in 8 bits with a scale per ``group`` = 32, 64 or 128 columns."""
    rt = _rt()
    T, K = _matrix(x, "x [T,K]")
    N = _columns(W, "W [K,N]")
    ty = x.dtype
    code = _code(rt, ty)
    pw = _tensor(W, (K, N), ty, x, "W [K,N]")
    pb = _tensor(bias, (N,), ty, x, "bias [N]") if bias is not None else 0
    if out_dtype is None:
        out_dtype = residual.dtype if residual is not None else y.dtype if y is not None else ty
    pr = _tensor(residual, (T, N), out_dtype, x, "residual") if residual is not None else 0
    save_code, save_group = _save_kind(rt, save, group, ty, code) if save is not None else (code, 0)
    sizes, need = _dense("fff_linear", T, K, N, code, _code(rt, out_dtype), _act_code(act),
                         save_code, save_group, code, 0, code)
    handle = _here(rt, x, stream)
    y, py = _output(rt, y, (T, N), out_dtype, x, "y", stream)
    pre, pp, ps = _saved(rt, save, group, (T, N), ty, x, stream) if save is not None else (None, 0, 0)
    workspace, pws, have = _workspace(rt, workspace, need, x, stream)
    st = (_lib or load_library()).fff_linear(sizes, x.data_ptr(), pw, pb, pr, py, pp, ps, pws, have,
                                             handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_linear")
    return Linear(y, pre)


def linear_backward(dy, x, W, *, act: str = "none", pre=None, want_dx: bool = True,
                    want_dW: bool = True, want_dbias: bool = False, grad_dtype=None, dx=None,
                    dW=None, dbias=None, workspace=None, stream=None) -> LinearGrad:
    """fff_linear_backward: the gradients of linear's inputs from dy [T,N]
    (which itself is the residual's).  ``x`` [T,K] is a tensor or a Checkpoint
    (None where dW is not wanted), ``pre`` what linear saved (a tensor or a
    Checkpoint; needed with an activation).  dW is float32, or of
    ``grad_dtype``; dbias is float32.  Outputs that are passed are filled."""
    rt = _rt()
    T, N = _matrix(dy, "dy [T,N]")
    K, _ = _matrix(W, "W [K,N]")
    ty = dy.dtype
    code, act_code = _code(rt, ty), _act_code(act)
    pw = _tensor(W, (K, N), ty, dy, "W [K,N]")
    px = pxs = pp = pps = pdx = pdw = pdb = x_group = save_group = 0
    x_code = save_code = code
    want_dx, want_dW = want_dx or dx is not None, want_dW or dW is not None
    if want_dW:
        if x is None:
            raise ValueError("dW needs x")
        px, pxs, x_code, x_group = _kept(rt, x, (T, K), ty, dy, "x [T,K]")
    if act_code:
        if pre is None:
            raise ValueError(f"act {act!r} needs what linear saved")
        pp, pps, save_code, save_group = _kept(rt, pre, (T, N), ty, dy, "pre [T,N]")
    grad_dtype = grad_dtype or (dW.dtype if dW is not None else rt.f32)
    sizes, need = _dense("fff_linear_backward", T, K, N, code, code, act_code, save_code, save_group,
                         x_code, x_group, _code(rt, grad_dtype))
    handle = _here(rt, dy, stream)
    if want_dx:
        dx, pdx = _output(rt, dx, (T, K), ty, dy, "dx", stream)
    if want_dW:
        dW, pdw = _output(rt, dW, (K, N), grad_dtype, dy, "dW", stream)
    if want_dbias or dbias is not None:
        dbias, pdb = _output(rt, dbias, (N,), rt.f32, dy, "dbias", stream)
    workspace, pws, have = _workspace(rt, workspace, need, dy, stream)
    st = (_lib or load_library()).fff_linear_backward(sizes, dy.data_ptr(), px, pxs, pw, pp, pps, pdx,
                                                      pdw, pdb, pws, have, handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_linear_backward")
    return LinearGrad(dx, dW, dbias)


def gated(x, W_gate, W_up, *, act: str = "silu", save: Optional[str] = None, group: int = 128, h=None,
          workspace=None, stream=None) -> Gated:
    """fff_gated: h = act(x . W_gate) * (x . W_up), x [T,d], weights [d,F], in
    one kernel.  ``save`` keeps both projections for gated_backward, as
    linear's does."""
    rt = _rt()
    T, d = _matrix(x, "x [T,d]")
    F = _columns(W_gate, "W_gate [d,F]")
    ty = x.dtype
    code = _code(rt, ty)
    pg = _tensor(W_gate, (d, F), ty, x, "W_gate [d,F]")
    pu = _tensor(W_up, (d, F), ty, x, "W_up [d,F]")
    save_code, save_group = _save_kind(rt, save, group, ty, code) if save is not None else (code, 0)
    sizes, need = _dense("fff_gated", T, d, F, code, code, _act_code(act), save_code, save_group, code,
                         0, code)
    handle = _here(rt, x, stream)
    h, ph = _output(rt, h, (T, F), ty, x, "h", stream)
    gate = up = None
    p0 = s0 = p1 = s1 = 0
    if save is not None:
        gate, p0, s0 = _saved(rt, save, group, (T, F), ty, x, stream)
        up, p1, s1 = _saved(rt, save, group, (T, F), ty, x, stream)
    workspace, pws, have = _workspace(rt, workspace, need, x, stream)
    st = (_lib or load_library()).fff_gated(sizes, x.data_ptr(), pg, pu, ph, p0, s0, p1, s1, pws, have,
                                            handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_gated")
    return Gated(h, gate, up)


def gated_backward(dh, x, W_gate, W_up, gate, up, *, act: str = "silu", want_dx: bool = True,
                   want_dW: bool = True, want_h: bool = False, grad_dtype=None, dx=None, dW_gate=None,
                   dW_up=None, h=None, workspace=None, stream=None) -> GatedGrad:
    """fff_gated_backward: the gradients of gated's inputs from dh [T,F].
    ``gate`` and ``up`` are what gated saved (tensors, or Checkpoints of one
    group), ``x`` [T,d] a tensor or a Checkpoint (None where the weights'
    gradients are not wanted).  ``want_h``: h made again from gate and up, for
    the product that follows.  The weights' gradients are float32, or of
    ``grad_dtype``.  Outputs that are passed are filled."""
    rt = _rt()
    T, F = _matrix(dh, "dh [T,F]")
    d, _ = _matrix(W_gate, "W_gate [d,F]")
    ty = dh.dtype
    code = _code(rt, ty)
    pg = _tensor(W_gate, (d, F), ty, dh, "W_gate [d,F]")
    pu = _tensor(W_up, (d, F), ty, dh, "W_up [d,F]")
    p0, s0, save_code, save_group = _kept(rt, gate, (T, F), ty, dh, "gate [T,F]")
    p1, s1, up_code, up_group = _kept(rt, up, (T, F), ty, dh, "up [T,F]")
    if (up_code, up_group) != (save_code, save_group):
        raise ValueError("gate and up must be kept alike")
    px = pxs = pdx = pdg = pdu = ph = x_group = 0
    x_code = code
    if (dW_gate is None) != (dW_up is None):
        raise ValueError("dW_gate and dW_up go together")
    want_dx, want_dW = want_dx or dx is not None, want_dW or dW_gate is not None
    if want_dW:
        if x is None:
            raise ValueError("the weights' gradients need x")
        px, pxs, x_code, x_group = _kept(rt, x, (T, d), ty, dh, "x [T,d]")
    grad_dtype = grad_dtype or (dW_gate.dtype if dW_gate is not None else rt.f32)
    sizes, need = _dense("fff_gated_backward", T, d, F, code, code, _act_code(act), save_code,
                         save_group, x_code, x_group, _code(rt, grad_dtype))
    handle = _here(rt, dh, stream)
    if want_dx:
        dx, pdx = _output(rt, dx, (T, d), ty, dh, "dx", stream)
    if want_dW:
        dW_gate, pdg = _output(rt, dW_gate, (d, F), grad_dtype, dh, "dW_gate", stream)
        dW_up, pdu = _output(rt, dW_up, (d, F), grad_dtype, dh, "dW_up", stream)
    if want_h or h is not None:
        h, ph = _output(rt, h, (T, F), ty, dh, "h", stream)
    workspace, pws, have = _workspace(rt, workspace, need, dh, stream)
    st = (_lib or load_library()).fff_gated_backward(sizes, dh.data_ptr(), px, pxs, pg, pu, p0, s0, p1,
                                                     s1, pdx, pdg, pdu, ph, pws, have, handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_gated_backward")
    return GatedGrad(dx, dW_gate, dW_up, h)


def checkpoint(x, group: int = 128, *, codes=None, scale=None, stream=None) -> Checkpoint:
    """fff_checkpoint_save: rows x [T,d] in 8 bits with a float32 scale for
    every ``group`` = 32, 64 or 128 columns, or (0) for the row."""
    rt = _rt()
    T, d = _matrix(x, "x [T,d]")
    code = _code(rt, x.dtype)
    if group not in (0, 32, 64, 128):
        raise FFFError(ERROR_INVALID_VALUE, f"checkpoint with group {group}")
    if d > DENSE_MAX_WIDTH:
        raise FFFError(ERROR_NOT_SUPPORTED, f"checkpoint of rows of {d} columns")
    handle = _here(rt, x, stream)
    codes, pc = _output(rt, codes, (T, d), rt.f8, x, "codes", stream)
    scale, ps = _output(rt, scale, _scales(T, d, group), rt.f32, x, "scale", stream)
    st = (_lib or load_library()).fff_checkpoint_save(T, d, code, group, x.data_ptr(), pc, ps, handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_checkpoint_save")
    return Checkpoint(codes, scale, group)


def restore(kept: Checkpoint, dtype=None, *, out=None, stream=None):
    """fff_checkpoint_load: the rows that a Checkpoint stands for, in ``dtype``
    (bf16 by default, or float32)."""
    rt = _rt()
    T, d = _matrix(kept.codes, "codes [T,d]")
    if d > DENSE_MAX_WIDTH:
        raise FFFError(ERROR_NOT_SUPPORTED, f"checkpoint of rows of {d} columns")
    pc, ps, _, group = _kept(rt, kept, (T, d), rt.f8, kept.codes, "kept")
    dtype = dtype or (out.dtype if out is not None else rt.bf16)
    code = _code(rt, dtype)
    handle = _here(rt, kept.codes, stream)
    out, po = _output(rt, out, (T, d), dtype, kept.codes, "out", stream)
    st = (_lib or load_library()).fff_checkpoint_load(T, d, code, group, pc, ps, po, handle)
    if st != SUCCESS:
        raise FFFError(st, "fff_checkpoint_load")
    return out
