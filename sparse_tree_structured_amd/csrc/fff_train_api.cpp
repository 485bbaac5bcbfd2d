// C ABI of the operators around the layer: the root-mean-square norm with its
// backward pass, the AdamW step and the gradient norm.  As for the layer
// itself, every argument is validated before any HIP call.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/fff.h"
#include "launch_train.hpp"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
// Workgroups of one launch: 256 threads each, and a launch has fewer than
// 2^32 threads.
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;
static_assert(fff::kNormSmallChunks <= fff::kNormMaxTensors, "a small list fits the arguments");
// One tensor of the optimiser fits one launch.
constexpr int64_t kMaxTensor = int64_t(1) << 34;
static_assert(kMaxTensor / fff::kAdamwChunk <= kMaxBlocks &&
                  (kMaxTensor >> 32) < (1 << (32 - fff::kFirstBits)) &&
                  kMaxBlocks < (1 << fff::kFirstBits),
              "a tensor fits a launch, and its descriptor the arguments");

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t type_size(int32_t dtype) {
  return dtype == FFF_DTYPE_F32 ? 4 : dtype == FFF_DTYPE_BF16 ? 2 : 1;
}

// An address that gfx950 can have.
bool in_space(const void* p) {
  return reinterpret_cast<uintptr_t>(p) >> fff::kAddressBits == 0;
}

// A pointer that a tensor of this type can have.
bool good(const void* p, int32_t dtype) { return p && aligned(p, type_size(dtype)); }
bool good_or_null(const void* p, int32_t dtype) { return aligned(p, type_size(dtype)); }

fff_status_t hip_status(hipError_t e) { return e == hipSuccess ? FFF_SUCCESS : FFF_ERROR_HIP; }

fff_status_t check_norm(const fff_norm_shape_t* s) {
  if (!s) return FFF_ERROR_INVALID_VALUE;
  if (s->dtype != FFF_DTYPE_F32 && s->dtype != FFF_DTYPE_BF16) return FFF_ERROR_NOT_SUPPORTED;
  if (s->stream_dtype != s->dtype && s->stream_dtype != FFF_DTYPE_F32)
    return FFF_ERROR_NOT_SUPPORTED;
  if (s->T < 0 || s->T > INT32_MAX || s->d <= 0 || s->T * s->d >= kMaxElems)
    return FFF_ERROR_INVALID_VALUE;
  if (s->d > fff::kNormMaxWidth) return FFF_ERROR_NOT_SUPPORTED;
  if (!(s->eps >= 0.0f) || !isfinite(s->eps) || !isfinite(s->weight_offset))
    return FFF_ERROR_INVALID_VALUE;
  return FFF_SUCCESS;
}

uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

// Key of tensor t's random numbers under a seed.
uint32_t random_key(uint64_t seed, uint32_t t) {
  return mix32(mix32(static_cast<uint32_t>(seed) ^ (0x9E3779B9u * (t + 1))) ^
               static_cast<uint32_t>(seed >> 32));
}

fff_status_t check_grads(const fff_adamw_tensor_t* tensors, int64_t count) {
  if (count < 0 || count > INT32_MAX || (count > 0 && !tensors)) return FFF_ERROR_INVALID_VALUE;
  for (int64_t i = 0; i < count; ++i) {
    const fff_adamw_tensor_t& t = tensors[i];
    if (t.grad_dtype != FFF_DTYPE_F32 && t.grad_dtype != FFF_DTYPE_BF16)
      return FFF_ERROR_NOT_SUPPORTED;
    if (t.n < 0 || t.n > kMaxTensor) return FFF_ERROR_INVALID_VALUE;
    if (t.n > 0 && !good(t.grad, t.grad_dtype)) return FFF_ERROR_INVALID_VALUE;
  }
  return FFF_SUCCESS;
}

int64_t grad_chunks(const fff_adamw_tensor_t* tensors, int64_t count, int chunk) {
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) n += (tensors[i].n + chunk - 1) / chunk;
  return n;
}

// Whether one workgroup takes all of the list.
bool grads_small(const fff_adamw_tensor_t* tensors, int64_t count) {
  return grad_chunks(tensors, count, fff::kNormSmallChunk) <= fff::kNormSmallChunks;
}

size_t grad_norm_bytes(const fff_adamw_tensor_t* tensors, int64_t count) {
  return grads_small(tensors, count)
             ? 0
             : size_t(grad_chunks(tensors, count, fff::kNormChunk)) * sizeof(double);
}

}  // namespace

extern "C" {

fff_status_t fff_rms_norm(const fff_norm_shape_t* shape, const void* x, const void* residual,
                          const void* weight, void* y, float* scale, void* residual_out,
                          float* rstd, hipStream_t stream) {
  fff_status_t st = check_norm(shape);
  if (st != FFF_SUCCESS) return st;
  const fff_norm_shape_t& s = *shape;
  if (s.out_dtype != s.dtype && s.out_dtype != FFF_DTYPE_E4M3) return FFF_ERROR_NOT_SUPPORTED;
  const bool e4m3 = s.out_dtype == FFF_DTYPE_E4M3;
  if (e4m3 ? s.group != 0 && s.group != 32 && s.group != 64 && s.group != 128 : s.group != 0)
    return FFF_ERROR_INVALID_VALUE;
  if (s.T == 0) return FFF_SUCCESS;
  if ((!x && !residual) || !good_or_null(x, s.dtype) || !good_or_null(residual, s.stream_dtype) ||
      !good_or_null(weight, s.dtype) || !good(y, s.out_dtype) ||
      !good_or_null(residual_out, s.stream_dtype) || !good_or_null(rstd, FFF_DTYPE_F32) ||
      (e4m3 && !good(scale, FFF_DTYPE_F32)))
    return FFF_ERROR_INVALID_VALUE;
  fff::NormArgs a;
  a.T = s.T;
  a.d = s.d;
  a.group = s.group;
  a.bf16 = s.dtype == FFF_DTYPE_BF16;
  a.stream_bf16 = s.stream_dtype == FFF_DTYPE_BF16;
  a.e4m3 = e4m3;
  a.eps = s.eps;
  a.weight_offset = s.weight_offset;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.y = y;
  a.scale = scale;
  a.residual_out = residual_out;
  a.rstd = rstd;
  return hip_status(fff::launch_rms_norm(a, stream));
}

fff_status_t fff_rms_norm_backward_workspace_size(const fff_norm_shape_t* shape, size_t* bytes) {
  fff_status_t st = check_norm(shape);
  if (st != FFF_SUCCESS) return st;
  if (!bytes) return FFF_ERROR_INVALID_VALUE;
  *bytes = fff::rms_norm_backward_partials(shape->T, shape->d, shape->dtype == FFF_DTYPE_BF16,
                                           shape->stream_dtype == FFF_DTYPE_BF16) *
           size_t(shape->d) * sizeof(float);
  return FFF_SUCCESS;
}

fff_status_t fff_rms_norm_backward(const fff_norm_shape_t* shape, const void* dy, const void* z,
                                   const void* weight, const float* rstd, const void* dresidual,
                                   void* dz, void* dx, float* dweight, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  fff_status_t st = fff_rms_norm_backward_workspace_size(shape, &need);
  if (st != FFF_SUCCESS) return st;
  const fff_norm_shape_t& s = *shape;
  if (!good_or_null(dweight, FFF_DTYPE_F32)) return FFF_ERROR_INVALID_VALUE;
  if (s.T > 0) {
    if (!good(dy, s.dtype) || !good(z, s.stream_dtype) || !good_or_null(weight, s.dtype) ||
        !good(rstd, FFF_DTYPE_F32) || !good_or_null(dresidual, s.stream_dtype) ||
        !good(dz, s.stream_dtype) || !good_or_null(dx, s.dtype))
      return FFF_ERROR_INVALID_VALUE;
    if (dweight && need > 0 && (!workspace || workspace_bytes < need)) return FFF_ERROR_WORKSPACE;
    if (!aligned(workspace, 256)) return FFF_ERROR_INVALID_VALUE;
  }
  if (s.T == 0 && !dweight) return FFF_SUCCESS;
  fff::NormGradArgs a;
  a.T = s.T;
  a.d = s.d;
  a.bf16 = s.dtype == FFF_DTYPE_BF16;
  a.stream_bf16 = s.stream_dtype == FFF_DTYPE_BF16;
  a.weight_offset = s.weight_offset;
  a.dy = dy;
  a.z = z;
  a.weight = weight;
  a.rstd = rstd;
  a.dresidual = dresidual;
  a.dz = dz;
  a.dx = dx;
  a.dweight = dweight;
  a.partial = dweight && need > 0 ? static_cast<float*>(workspace) : nullptr;
  return hip_status(fff::launch_rms_norm_backward(a, stream));
}

fff_status_t fff_adamw_step(const fff_adamw_config_t* config, const fff_adamw_tensor_t* tensors,
                            int64_t count, hipStream_t stream) {
  if (!config) return FFF_ERROR_INVALID_VALUE;
  const fff_adamw_config_t& c = *config;
  if (c.state_dtype != FFF_DTYPE_F32 && c.state_dtype != FFF_DTYPE_E4M3)
    return FFF_ERROR_NOT_SUPPORTED;
  const bool e4m3 = c.state_dtype == FFF_DTYPE_E4M3;
  if (!isfinite(c.lr) || !(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0) ||
      !(c.eps >= 0.0) || !isfinite(c.eps) || c.step < 1 ||
      !good_or_null(c.grad_scale, FFF_DTYPE_F32))
    return FFF_ERROR_INVALID_VALUE;
  fff_status_t st = check_grads(tensors, count);
  if (st != FFF_SUCCESS) return st;
  // Tensors of one kind (weights' and gradients' types) share launches.
  constexpr int kKinds = 6;
  bool any[kKinds] = {};
  auto kind_of = [](const fff_adamw_tensor_t& t) {
    const int p = t.param_dtype == FFF_DTYPE_F32 ? fff::kParamF32
                  : t.master                     ? fff::kParamMaster
                                                 : fff::kParamBf16;
    return 2 * p + (t.grad_dtype == FFF_DTYPE_BF16 ? 1 : 0);
  };
  for (int64_t i = 0; i < count; ++i) {
    const fff_adamw_tensor_t& t = tensors[i];
    if (t.param_dtype != FFF_DTYPE_F32 && t.param_dtype != FFF_DTYPE_BF16)
      return FFF_ERROR_NOT_SUPPORTED;
    if (t.master && t.param_dtype != FFF_DTYPE_BF16) return FFF_ERROR_NOT_SUPPORTED;
    if (!isfinite(t.lr_scale) || !isfinite(t.weight_decay)) return FFF_ERROR_INVALID_VALUE;
    if (t.n == 0) continue;
    if (!good(t.param, t.param_dtype) || !good_or_null(t.master, FFF_DTYPE_F32) ||
        !good(t.exp_avg, c.state_dtype) || !good(t.exp_avg_sq, c.state_dtype) ||
        (e4m3 && !(t.scale && aligned(t.scale, 8))) || !in_space(t.param) || !in_space(t.master) ||
        !in_space(t.grad) || !in_space(t.exp_avg) || !in_space(t.exp_avg_sq) || !in_space(t.scale))
      return FFF_ERROR_INVALID_VALUE;
    any[kind_of(t)] = true;
  }
  fff::AdamwArgs a;
  a.beta1 = static_cast<float>(c.beta1);
  a.one_beta1 = static_cast<float>(1.0 - c.beta1);
  a.beta2 = static_cast<float>(c.beta2);
  a.one_beta2 = static_cast<float>(1.0 - c.beta2);
  a.eps = static_cast<float>(c.eps);
  a.long_m = fff::adamw_long_m(a.eps);
  a.root = static_cast<float>(1.0 / sqrt(1.0 - pow(c.beta2, static_cast<double>(c.step))));
  a.grad_scale = c.grad_scale;
  const double bias1 = 1.0 - pow(c.beta1, static_cast<double>(c.step));
  for (int kind = 0; kind < kKinds; ++kind) {
    if (!any[kind]) continue;
    int64_t blocks = 0;
    a.count = 0;
    auto flush = [&]() {
      if (a.count == 0) return hipSuccess;
      const hipError_t e = fff::launch_adamw(a, static_cast<int>(blocks), kind / 2, kind % 2 != 0,
                                             e4m3, c.stochastic != 0, stream);
      a.count = 0;
      blocks = 0;
      return e;
    };
    for (int64_t i = 0; i < count; ++i) {
      const fff_adamw_tensor_t& t = tensors[i];
      if (t.n == 0 || kind_of(t) != kind) continue;
      const int64_t need = (t.n + fff::kAdamwChunk - 1) / fff::kAdamwChunk;
      if ((a.count == fff::kAdamwMaxTensors || blocks + need > kMaxBlocks) && flush() != hipSuccess)
        return FFF_ERROR_HIP;
      using E = fff::AdamwEntry;
      a.first[a.count] = static_cast<uint32_t>(blocks) |
                         static_cast<uint32_t>(t.n >> 32) << fff::kFirstBits;
      E& e = a.e[a.count++];
      e.set(E::kParam, t.param);
      e.set(E::kMaster, t.master);
      e.set(E::kGrad, t.grad);
      e.set(E::kExpAvg, t.exp_avg);
      e.set(E::kExpAvgSq, t.exp_avg_sq);
      e.set(E::kScale, t.scale);
      e.n_lo = static_cast<uint32_t>(t.n);
      e.key = random_key(c.seed, static_cast<uint32_t>(i));
      const double lr = c.lr * t.lr_scale;
      e.decay = static_cast<float>(1.0 - lr * t.weight_decay);
      e.step = static_cast<float>(lr / bias1);
      blocks += need;
    }
    if (flush() != hipSuccess) return FFF_ERROR_HIP;
  }
  return FFF_SUCCESS;
}

fff_status_t fff_grad_norm_workspace_size(const fff_adamw_tensor_t* tensors, int64_t count,
                                          size_t* bytes) {
  fff_status_t st = check_grads(tensors, count);
  if (st != FFF_SUCCESS) return st;
  if (!bytes) return FFF_ERROR_INVALID_VALUE;
  *bytes = grad_norm_bytes(tensors, count);
  return FFF_SUCCESS;
}

fff_status_t fff_grad_norm(const fff_adamw_tensor_t* tensors, int64_t count, double max_norm,
                           float* out, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  fff_status_t st = check_grads(tensors, count);
  if (st != FFF_SUCCESS) return st;
  if (!(max_norm > 0.0) || !good(out, FFF_DTYPE_F32)) return FFF_ERROR_INVALID_VALUE;
  const size_t need_bytes = grad_norm_bytes(tensors, count);
  if (need_bytes > 0 && (!workspace || workspace_bytes < need_bytes)) return FFF_ERROR_WORKSPACE;
  if (!aligned(workspace, 256)) return FFF_ERROR_INVALID_VALUE;
  const bool small = grads_small(tensors, count);
  const int chunk = small ? fff::kNormSmallChunk : fff::kNormChunk;
  double* partial = static_cast<double*>(workspace);
  fff::GradNormArgs a;
  int64_t blocks = 0, done = 0;
  a.count = 0;
  auto flush = [&]() {
    if (a.count == 0) return hipSuccess;
    a.partial = partial + done;
    const hipError_t e = fff::launch_grad_squares(a, static_cast<int>(blocks), stream);
    done += blocks;
    a.count = 0;
    blocks = 0;
    return e;
  };
  for (int64_t i = 0; i < count; ++i) {
    const fff_adamw_tensor_t& t = tensors[i];
    if (t.n == 0) continue;
    const int64_t need = (t.n + chunk - 1) / chunk;
    if ((a.count == fff::kNormMaxTensors || blocks + need > kMaxBlocks) && flush() != hipSuccess)
      return FFF_ERROR_HIP;
    a.first[a.count] = static_cast<uint32_t>(blocks);
    fff::GradEntry& e = a.e[a.count++];
    e.grad = t.grad;
    e.n = t.grad_dtype == FFF_DTYPE_BF16 ? -t.n : t.n;
    blocks += need;
  }
  if (small)  // at most one tensor to a chunk: the list fits the arguments
    return hip_status(fff::launch_grad_norm_small(a, static_cast<uint32_t>(blocks), max_norm, out,
                                                  stream));
  if (flush() != hipSuccess) return FFF_ERROR_HIP;
  return hip_status(fff::launch_grad_norm_final(partial, done, max_norm, out, stream));
}

}  // extern "C"
