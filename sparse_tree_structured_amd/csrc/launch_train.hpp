// Host-side launchers of the kernels around the layer: the norm with its
// backward pass, the optimiser step and the gradient norm.  Each enqueues its
// kernel(s) on `st` and returns hipGetLastError().  Arguments have been
// validated by the C-ABI layer before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fff {

constexpr int kNormMaxWidth = 32768;  // a row is held in one workgroup's registers

struct NormArgs {
  int64_t T;
  int d;
  int group;          // e4m3: columns per scale, 0 = the row
  bool bf16;          // layer type (x, weight, y)
  bool stream_bf16;   // residual, residual_out
  bool e4m3;          // y in 8 bits
  float eps, weight_offset;
  const void *x, *residual, *weight;
  void* y;
  float* scale;
  void* residual_out;
  float* rstd;
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t st);

struct NormGradArgs {
  int64_t T;
  int d;
  bool bf16, stream_bf16;
  float weight_offset;
  const void *dy, *z, *weight;
  const float* rstd;
  const void* dresidual;
  void *dz, *dx;
  float *dweight, *partial;
  int rows;  // rows and columns in one launch: workgroups of rows (set by the launcher)
};
// Rows of d floats in the workspace.
size_t rms_norm_backward_partials(int64_t T, int d, bool bf16, bool stream_bf16);
hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t st);

// ---- optimiser ----

constexpr int kStateBlock = 128;      // elements per scale of an 8-bit state
constexpr int kAdamwChunk = 2048;     // elements per workgroup
constexpr int kAdamwMaxTensors = 72;  // descriptors that fit a kernel's arguments (4 KB)

// One tensor.  Every launch has a tail of a few microseconds in which the
// last workgroups compute and nothing loads, so as many tensors as possible
// go into one: addresses are kept in gfx950's 48 bits.
struct AdamwEntry {
  enum { kParam, kMaster, kGrad, kExpAvg, kExpAvgSq, kScale, kPointers };
  uint32_t lo[kPointers];
  uint16_t hi[kPointers];
  uint32_t n_lo;  // elements: low half (the high bits are in AdamwArgs::first)
  float decay;    // 1 - lr weight_decay
  float step;     // lr / (1 - beta1^t)
  uint32_t key;   // of its random numbers

  void set(int which, const void* p) {
    lo[which] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
    hi[which] = static_cast<uint16_t>(reinterpret_cast<uintptr_t>(p) >> 32);
  }
  // By way of a global pointer, or the compiler takes the accesses for
  // flat ones.
  template <typename T> __device__ T* get(int which) const {
    return (T*)(__attribute__((address_space(1))) T*)(
        static_cast<uintptr_t>(lo[which]) | static_cast<uintptr_t>(hi[which]) << 32);
  }
};
constexpr int kAddressBits = 48;
constexpr int kFirstBits = 24;  // workgroups of a launch: below 2^24

struct AdamwArgs {
  float beta1, one_beta1, beta2, one_beta2, eps, root;  // root: 1 / sqrt(1 - beta2^t)
  const float* grad_scale;
  uint32_t long_m;  // adamw_long_m(eps)
  int count;
  // Each tensor's first workgroup (24 bits) and, above it, its n >> 32.
  uint32_t first[kAdamwMaxTensors];
  AdamwEntry e[kAdamwMaxTensors];
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

// The largest 2 bits(m) - 1 (zero wraps to the top) that needs the long
// quotient m / (sqrt(v) / sqrt(1 - beta2^t) + eps): the short one is for
// m = 0 and m from 2^-60 on, over divisors in [2^-60, 2^90).  A root in its
// own short range is below 2^30 and 1 / sqrt(1 - beta2^t) below 2^27 for
// every beta2 below 1, so eps in [2^-60, 2^60) gives such a divisor; beside
// any other every m takes the long quotient.
constexpr uint32_t adamw_long_m(float eps) {
  return eps >= 0x1p-60f && eps < 0x1p60f ? 2 * (67u << 23) - 2 : ~0u;
}

enum AdamwParam { kParamF32 = 0, kParamBf16 = 1, kParamMaster = 2 };

// From this many bytes on a launch reads and writes past the caches: nothing
// of it is used again before the next step.  A layer's 17.2 M elements with
// masters take 86.6 us instead of 97.2 (8-bit states: 54.2 and 60.1), 195 MB
// 34.6 instead of 35.9; 97 MB, which the 256 MB last-level cache can hold for
// the next reader, 19.3 instead of 16.7, and 117 MB 23.4 instead of 21.5.
constexpr int64_t kStreamBytes = int64_t(160) << 20;

// Whether a launch of this many workgroups does.
constexpr bool adamw_streams(int blocks, int param, bool grad_bf16, bool state_e4m3) {
  const int64_t each = (param == kParamF32 ? 8 : param == kParamBf16 ? 4 : 10) +
                       (grad_bf16 ? 2 : 4) + (state_e4m3 ? 4 : 16);
  return int64_t(blocks) * kAdamwChunk * each >= kStreamBytes;
}

hipError_t launch_adamw(const AdamwArgs& a, int blocks, int param, bool grad_bf16, bool state_e4m3,
                        bool stochastic, hipStream_t st);

constexpr int kNormChunk = 16384;     // gradient elements per workgroup
constexpr int kNormSmallChunk = 2048;  // per wavefront, for a small list
constexpr int kNormSmallChunks = 64;   // of at most so many of these
constexpr int kNormMaxTensors = 192;

struct GradEntry {
  const void* grad;
  int64_t n;         // elements; negative: bf16
};

struct GradNormArgs {
  double* partial;   // one per workgroup
  int count;
  uint32_t first[kNormMaxTensors];
  GradEntry e[kNormMaxTensors];
};
static_assert(sizeof(GradNormArgs) <= 4096, "kernel arguments");

hipError_t launch_grad_squares(const GradNormArgs& a, int blocks, hipStream_t st);
hipError_t launch_grad_norm_small(const GradNormArgs& a, uint32_t chunks, double max_norm, float* out,
                                  hipStream_t st);
hipError_t launch_grad_norm_final(const double* partial, int64_t count, double max_norm, float* out,
                                  hipStream_t st);

}  // namespace fff
