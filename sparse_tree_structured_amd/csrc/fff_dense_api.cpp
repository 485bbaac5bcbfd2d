// C ABI of the dense feed-forward block: the product with an epilogue, the
// gated pair, their backward passes, and 8-bit checkpoints.  As for the layer
// itself, every argument is validated before any HIP call.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "../../include/fff.h"
#include "launch_dense.hpp"

namespace {

using fff::Product;
using Shape = fff_dense_shape_t;

constexpr int64_t kMaxElems = int64_t(1) << 40;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t type_size(int32_t dtype) {
  return dtype == FFF_DTYPE_F32 ? 4 : dtype == FFF_DTYPE_BF16 ? 2 : 1;
}
bool good(const void* p, int32_t dtype) { return p && aligned(p, type_size(dtype)); }
bool good_or_null(const void* p, int32_t dtype) { return aligned(p, type_size(dtype)); }

fff_status_t hip_status(hipError_t e) { return e == hipSuccess ? FFF_SUCCESS : FFF_ERROR_HIP; }

bool layer_type(int32_t dtype) { return dtype == FFF_DTYPE_F32 || dtype == FFF_DTYPE_BF16; }

// A tensor of the layer's type, or in 8 bits by groups.
fff_status_t check_kept(int32_t dtype, int32_t group, int32_t layer, bool row_scale) {
  if (dtype != layer && dtype != FFF_DTYPE_E4M3) return FFF_ERROR_NOT_SUPPORTED;
  if (dtype != FFF_DTYPE_E4M3) return group == 0 ? FFF_SUCCESS : FFF_ERROR_INVALID_VALUE;
  if (group == 32 || group == 64 || group == 128 || (group == 0 && row_scale)) return FFF_SUCCESS;
  return FFF_ERROR_INVALID_VALUE;
}

fff_status_t check_shape(const Shape* s, bool backward, bool gated) {
  if (!s) return FFF_ERROR_INVALID_VALUE;
  if (!layer_type(s->dtype)) return FFF_ERROR_NOT_SUPPORTED;
  if (s->T < 0 || s->T > INT32_MAX || s->K <= 0 || s->N <= 0) return FFF_ERROR_INVALID_VALUE;
  if (s->K > FFF_DENSE_MAX_WIDTH || s->N > FFF_DENSE_MAX_WIDTH) return FFF_ERROR_NOT_SUPPORTED;
  if (s->T * s->K >= kMaxElems || s->T * s->N >= kMaxElems || int64_t(s->K) * s->N >= kMaxElems)
    return FFF_ERROR_INVALID_VALUE;
  if (s->act < FFF_ACT_NONE || s->act > FFF_ACT_RELU) return FFF_ERROR_INVALID_VALUE;
  fff_status_t st = check_kept(s->save_dtype, s->save_group, s->dtype, backward);
  if (st != FFF_SUCCESS) return st;
  if (backward) {
    st = check_kept(s->x_dtype, s->x_group, s->dtype, true);
    if (st != FFF_SUCCESS) return st;
    if (s->grad_dtype != FFF_DTYPE_F32 && s->grad_dtype != s->dtype) return FFF_ERROR_NOT_SUPPORTED;
  } else if (s->out_dtype != s->dtype && (gated || s->out_dtype != FFF_DTYPE_F32)) {
    return FFF_ERROR_NOT_SUPPORTED;
  }
  return FFF_SUCCESS;
}

size_t padded(size_t bytes) { return (bytes + 255) & ~size_t(255); }

// The products of a shape, without pointers: their sizes decide their workspace.
Product base(const Shape& s, fff::ProductKind kind, fff::ProductPair pair) {
  Product p = {};
  p.kind = kind;
  p.pair = pair;
  p.bf16 = s.dtype == FFF_DTYPE_BF16;
  return p;
}

// x . W, or the gated pair's two.
Product forward_product(const Shape& s, bool gated) {
  Product p = base(s, fff::kProductNN, gated ? fff::kPairColumns : fff::kSingle);
  p.out_bf16 = s.out_dtype == FFF_DTYPE_BF16;
  p.lda = s.K;
  p.ldb = s.N;
  p.M = s.T;
  p.N = s.N;
  p.K = s.K;
  p.e.M = p.M;
  p.e.N = p.N;
  p.e.act = s.act;
  return p;
}

// Rows of N as the workspace holds them: whole 16-byte pieces.
int64_t da_ld(const Shape& s, bool gated) {
  return gated || s.act != FFF_ACT_NONE ? fff::planes_ld(s.N) : s.N;
}

// da . W^T (gated: two, one matrix after the other).
Product dx_product(const Shape& s, bool gated) {
  Product p = base(s, fff::kProductNT, gated ? fff::kPairSum : fff::kSingle);
  p.out_bf16 = p.bf16;
  p.lda = da_ld(s, gated);
  p.a_second = s.T * p.lda;
  p.ldb = s.N;
  p.M = s.T;
  p.N = s.K;
  p.K = s.N;
  p.e.M = p.M;
  p.e.N = p.N;
  return p;
}

// x^T . da (gated: two).
Product dw_product(const Shape& s, bool gated) {
  Product p = base(s, fff::kProductTN, gated ? fff::kPairTwo : fff::kSingle);
  p.out_bf16 = s.grad_dtype == FFF_DTYPE_BF16;
  p.lda = s.x_dtype == FFF_DTYPE_E4M3 ? fff::planes_ld(s.K) : s.K;
  p.ldb = da_ld(s, gated);
  p.M = s.K;
  p.N = s.N;
  p.K = s.T;
  p.e.M = p.M;
  p.e.N = p.N;
  return p;
}

// The backward passes' workspace.
struct Layout {
  size_t da, x, strips, planes, products, bytes;  // offsets, and all of it
};

// Whether da is needed in planes, too: float32 products large enough.
bool split_da(const Shape& s, bool gated) {
  return fff::split_wanted(dx_product(s, gated)) || fff::split_wanted(dw_product(s, gated));
}

// da's planes (gated: the gate's, then up's) from `at` on, in both products.
void give_planes(const Shape& s, bool gated, unsigned char* at, Product& dx, Product& dw) {
  if (!split_da(s, gated)) return;
  const int64_t ld = fff::planes_ld(s.N), plane = s.T * ld;
  dx.a_planes = dw.b_planes[0] = {at, ld, plane};
  dx.a_planes_second = 3 * plane;
  if (gated) dw.b_planes[1] = {at ? at + 6 * plane : nullptr, ld, plane};
}

Layout backward_layout(const Shape& s, bool gated) {
  const size_t e = type_size(s.dtype);
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += padded(bytes);
    return here;
  };
  const size_t rows = static_cast<size_t>(s.T);
  const size_t row = size_t(da_ld(s, gated)) * e;
  l.da = take(gated ? 2 * rows * row : s.act != FFF_ACT_NONE ? rows * row : 0);
  l.x = take(s.x_dtype == FFF_DTYPE_E4M3 ? rows * fff::planes_ld(s.K) * e : 0);
  l.strips = take(gated ? 0 : fff::act_backward_partials(s.T, s.N, s.dtype == FFF_DTYPE_BF16) * 4);
  // (the word of values beyond the planes, then the planes)
  l.planes = take(split_da(s, gated) ? 256 + (gated ? 2 : 1) * fff::planes_bytes(s.T, s.N) : 0);
  Product px = dx_product(s, gated), pw = dw_product(s, gated);
  give_planes(s, gated, nullptr, px, pw);
  const size_t dx = fff::product_workspace(px);
  const size_t dw = fff::product_workspace(pw);
  l.products = take(dx > dw ? dx : dw);
  l.bytes = at;
  return l;
}

fff_status_t check_fits(const Product& p) {
  return fff::product_fits(p) ? FFF_SUCCESS : FFF_ERROR_NOT_SUPPORTED;
}

fff_status_t forward_size(const Shape* s, bool gated, size_t* bytes) {
  fff_status_t st = check_shape(s, false, gated);
  if (st != FFF_SUCCESS) return st;
  const Product p = forward_product(*s, gated);
  st = check_fits(p);
  if (st != FFF_SUCCESS) return st;
  if (!bytes) return FFF_ERROR_INVALID_VALUE;
  *bytes = s->T == 0 ? 0 : fff::product_workspace(p);
  return FFF_SUCCESS;
}

fff_status_t backward_size(const Shape* s, bool gated, size_t* bytes) {
  fff_status_t st = check_shape(s, true, gated);
  if (st != FFF_SUCCESS) return st;
  st = check_fits(dx_product(*s, gated));
  if (st == FFF_SUCCESS) st = check_fits(dw_product(*s, gated));
  if (st != FFF_SUCCESS) return st;
  if (!bytes) return FFF_ERROR_INVALID_VALUE;
  *bytes = s->T == 0 ? 0 : backward_layout(*s, gated).bytes;
  return FFF_SUCCESS;
}

fff_status_t check_workspace(const void* workspace, size_t have, size_t need) {
  if (need > 0 && (!workspace || have < need)) return FFF_ERROR_WORKSPACE;
  return aligned(workspace, 256) ? FFF_SUCCESS : FFF_ERROR_INVALID_VALUE;
}

// Saved sums: a pointer of its type, and scales where they are in 8 bits.
bool good_save(const Shape& s, const void* save, const float* scale) {
  if (!good(save, s.save_dtype)) return false;
  return s.save_dtype != FFF_DTYPE_E4M3 || good(scale, FFF_DTYPE_F32);
}

void set_save(const Shape& s, Product& p, int which, void* save, float* scale) {
  p.e.save[which] = save;
  p.e.scale[which] = save && s.save_dtype == FFF_DTYPE_E4M3 ? scale : nullptr;
  p.e.group = s.save_group;
}

// The elementwise step and both products.
struct Backward {
  const void *dy, *x;
  const float* x_scale;
  const void *W[2], *save[2];
  const float* scale[2];
  void *dx, *dW[2], *h;
  float* dbias;
};

fff_status_t backward(const Shape& s, bool gated, const Backward& b, unsigned char* ws,
                      hipStream_t stream) {
  const Layout l = s.T == 0 ? Layout() : backward_layout(s, gated);
  const bool products = b.dx || b.dW[0];
  const bool own_da = gated || s.act != FFF_ACT_NONE;
  const void* da = own_da ? ws + l.da : b.dy;
  hipError_t e = hipSuccess;
  Product px = dx_product(s, gated), pw = dw_product(s, gated);
  const bool split = products && s.T > 0 && split_da(s, gated);
  if (split) {
    e = fff::start_word(ws + l.planes, stream, px.bad);
    if (e != hipSuccess) return FFF_ERROR_HIP;
    pw.bad = px.bad;
    give_planes(s, gated, ws + l.planes + 256, px, pw);
    if (!own_da) {
      e = fff::launch_split(b.dy, s.T, s.N, s.N, px.a_planes, px.bad, stream);
      if (e != hipSuccess) return FFF_ERROR_HIP;
    }
  }
  const bool restored = b.dW[0] && s.x_dtype == FFF_DTYPE_E4M3 && s.T > 0;
  if ((own_da && products && s.T > 0) || (b.h && s.T > 0) || b.dbias || restored) {
    fff::ActBackward a = {};
    if (restored) a.x = {s.T, s.K, s.x_group, b.x, b.x_scale, ws + l.x, fff::planes_ld(s.K)};
    a.T = s.T;
    a.N = s.N;
    a.bf16 = s.dtype == FFF_DTYPE_BF16;
    a.gated = gated;
    a.act = s.act;
    a.dy = b.dy;
    if (own_da) {
      for (int i = 0; i < 2; ++i) {
        a.save[i] = b.save[i];
        a.scale[i] = s.save_dtype == FFF_DTYPE_E4M3 ? b.scale[i] : nullptr;
      }
      a.group = s.save_group ? s.save_group : s.N;
      a.da = products ? ws + l.da : nullptr;
      a.da_ld = da_ld(s, gated);
      if (split) {
        a.da_planes[0] = pw.b_planes[0];
        a.da_planes[1] = pw.b_planes[1];
        a.bad = px.bad;
      }
    }
    a.h = b.h;
    a.dbias = b.dbias;
    a.partial = b.dbias ? reinterpret_cast<float*>(ws + l.strips) : nullptr;
    e = fff::launch_act_backward(a, stream);
    if (e != hipSuccess) return FFF_ERROR_HIP;
  }
  const size_t second = size_t(s.T) * da_ld(s, gated) * type_size(s.dtype);
  if (b.dx && s.T > 0) {
    px.a = da;
    px.b[0] = b.W[0];
    px.b[1] = b.W[1];
    px.e.out[0] = b.dx;
    e = fff::launch_product(px, ws + l.products, stream);
    if (e != hipSuccess) return FFF_ERROR_HIP;
  }
  if (b.dW[0]) {
    pw.a = restored ? ws + l.x : b.x;
    pw.b[0] = da;
    if (gated) pw.b[1] = static_cast<const unsigned char*>(da) + second;
    pw.e.out[0] = b.dW[0];
    pw.e.out[1] = b.dW[1];
    e = fff::launch_product(pw, ws + l.products, stream);
    if (e != hipSuccess) return FFF_ERROR_HIP;
  }
  return FFF_SUCCESS;
}

fff_status_t check_checkpoint(int64_t T, int32_t d, int32_t dtype, int32_t group, const void* x,
                              const void* codes, const float* scale) {
  if (!layer_type(dtype)) return FFF_ERROR_NOT_SUPPORTED;
  if (T < 0 || T > INT32_MAX || d <= 0 || T * d >= kMaxElems) return FFF_ERROR_INVALID_VALUE;
  if (d > FFF_DENSE_MAX_WIDTH) return FFF_ERROR_NOT_SUPPORTED;
  if (group != 0 && group != 32 && group != 64 && group != 128) return FFF_ERROR_INVALID_VALUE;
  if (T > 0 && (!good(x, dtype) || !codes || !good(scale, FFF_DTYPE_F32)))
    return FFF_ERROR_INVALID_VALUE;
  return FFF_SUCCESS;
}

}  // namespace

extern "C" {

fff_status_t fff_linear_workspace_size(const fff_dense_shape_t* shape, size_t* bytes) {
  return forward_size(shape, false, bytes);
}

fff_status_t fff_linear(const fff_dense_shape_t* shape, const void* x, const void* W,
                        const void* bias, const void* residual, void* y, void* pre,
                        float* pre_scale, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  size_t need = 0;
  fff_status_t st = forward_size(shape, false, &need);
  if (st != FFF_SUCCESS) return st;
  const Shape& s = *shape;
  if (s.T == 0) return FFF_SUCCESS;
  if (!good(x, s.dtype) || !good(W, s.dtype) || !good_or_null(bias, s.dtype) ||
      !good_or_null(residual, s.out_dtype) || !good(y, s.out_dtype) ||
      (pre && !good_save(s, pre, pre_scale)))
    return FFF_ERROR_INVALID_VALUE;
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != FFF_SUCCESS) return st;
  Product p = forward_product(s, false);
  p.a = x;
  p.b[0] = W;
  p.e.bias = bias;
  p.e.residual = residual;
  p.e.out[0] = y;
  set_save(s, p, 0, pre, pre_scale);
  return hip_status(fff::launch_product(p, workspace, stream));
}

fff_status_t fff_linear_backward_workspace_size(const fff_dense_shape_t* shape, size_t* bytes) {
  return backward_size(shape, false, bytes);
}

fff_status_t fff_linear_backward(const fff_dense_shape_t* shape, const void* dy, const void* x,
                                 const float* x_scale, const void* W, const void* pre,
                                 const float* pre_scale, void* dx, void* dW, float* dbias,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  fff_status_t st = backward_size(shape, false, &need);
  if (st != FFF_SUCCESS) return st;
  const Shape& s = *shape;
  if (!good_or_null(dx, s.dtype) || !good_or_null(dW, s.grad_dtype) ||
      !good_or_null(dbias, FFF_DTYPE_F32))
    return FFF_ERROR_INVALID_VALUE;
  if (!dx && !dW && !dbias) return FFF_SUCCESS;
  if (s.T > 0) {
    if (!good(dy, s.dtype) || (s.act != FFF_ACT_NONE && !good_save(s, pre, pre_scale)) ||
        (dx && !good(W, s.dtype)) ||
        (dW && (!good(x, s.x_dtype) ||
                (s.x_dtype == FFF_DTYPE_E4M3 && !good(x_scale, FFF_DTYPE_F32)))))
      return FFF_ERROR_INVALID_VALUE;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != FFF_SUCCESS) return st;
  }
  Backward b = {};
  b.dy = dy;
  b.x = x;
  b.x_scale = x_scale;
  b.W[0] = W;
  b.save[0] = pre;
  b.scale[0] = pre_scale;
  b.dx = dx;
  b.dW[0] = dW;
  b.dbias = dbias;
  return backward(s, false, b, static_cast<unsigned char*>(workspace), stream);
}

fff_status_t fff_gated_workspace_size(const fff_dense_shape_t* shape, size_t* bytes) {
  return forward_size(shape, true, bytes);
}

fff_status_t fff_gated(const fff_dense_shape_t* shape, const void* x, const void* W_gate,
                       const void* W_up, void* h, void* gate, float* gate_scale, void* up,
                       float* up_scale, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  size_t need = 0;
  fff_status_t st = forward_size(shape, true, &need);
  if (st != FFF_SUCCESS) return st;
  const Shape& s = *shape;
  if (s.T == 0) return FFF_SUCCESS;
  if (!good(x, s.dtype) || !good(W_gate, s.dtype) || !good(W_up, s.dtype) || !good(h, s.dtype) ||
      (gate && !good_save(s, gate, gate_scale)) || (up && !good_save(s, up, up_scale)))
    return FFF_ERROR_INVALID_VALUE;
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != FFF_SUCCESS) return st;
  Product p = forward_product(s, true);
  p.a = x;
  p.b[0] = W_gate;
  p.b[1] = W_up;
  p.e.out[0] = h;
  set_save(s, p, 0, gate, gate_scale);
  set_save(s, p, 1, up, up_scale);
  return hip_status(fff::launch_product(p, workspace, stream));
}

fff_status_t fff_gated_backward_workspace_size(const fff_dense_shape_t* shape, size_t* bytes) {
  return backward_size(shape, true, bytes);
}

fff_status_t fff_gated_backward(const fff_dense_shape_t* shape, const void* dh, const void* x,
                                const float* x_scale, const void* W_gate, const void* W_up,
                                const void* gate, const float* gate_scale, const void* up,
                                const float* up_scale, void* dx, void* dW_gate, void* dW_up,
                                void* h, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  size_t need = 0;
  fff_status_t st = backward_size(shape, true, &need);
  if (st != FFF_SUCCESS) return st;
  const Shape& s = *shape;
  if (!good_or_null(dx, s.dtype) || !good_or_null(dW_gate, s.grad_dtype) ||
      !good_or_null(dW_up, s.grad_dtype) || !good_or_null(h, s.dtype) || !dW_gate != !dW_up)
    return FFF_ERROR_INVALID_VALUE;
  if (!dx && !dW_gate && !h) return FFF_SUCCESS;
  if (s.T > 0) {
    if (!good(dh, s.dtype) || !good_save(s, gate, gate_scale) || !good_save(s, up, up_scale) ||
        (dx && (!good(W_gate, s.dtype) || !good(W_up, s.dtype))) ||
        (dW_gate && (!good(x, s.x_dtype) ||
                     (s.x_dtype == FFF_DTYPE_E4M3 && !good(x_scale, FFF_DTYPE_F32)))))
      return FFF_ERROR_INVALID_VALUE;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != FFF_SUCCESS) return st;
  }
  Backward b = {};
  b.dy = dh;
  b.x = x;
  b.x_scale = x_scale;
  b.W[0] = W_gate;
  b.W[1] = W_up;
  b.save[0] = gate;
  b.save[1] = up;
  b.scale[0] = gate_scale;
  b.scale[1] = up_scale;
  b.dx = dx;
  b.dW[0] = dW_gate;
  b.dW[1] = dW_up;
  b.h = h;
  return backward(s, true, b, static_cast<unsigned char*>(workspace), stream);
}

fff_status_t fff_checkpoint_save(int64_t T, int32_t d, int32_t dtype, int32_t group, const void* x,
                                 void* codes, float* scale, hipStream_t stream) {
  const fff_status_t st = check_checkpoint(T, d, dtype, group, x, codes, scale);
  if (st != FFF_SUCCESS || T == 0) return st;
  return hip_status(
      fff::launch_checkpoint_save(T, d, dtype == FFF_DTYPE_BF16, group, x, codes, scale, stream));
}

fff_status_t fff_checkpoint_load(int64_t T, int32_t d, int32_t dtype, int32_t group,
                                 const void* codes, const float* scale, void* x,
                                 hipStream_t stream) {
  const fff_status_t st = check_checkpoint(T, d, dtype, group, x, codes, scale);
  if (st != FFF_SUCCESS || T == 0) return st;
  return hip_status(
      fff::launch_checkpoint_load(T, d, dtype == FFF_DTYPE_BF16, group, codes, scale, x, stream));
}

}  // extern "C"
