// AdamW over many tensors in one launch, with moments in 32 or in 8 bits, and
// the gradient's norm over many tensors.
//
// Per element, with g already times *grad_scale:
//   m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr wd) - (lr / (1 - beta1^t)) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// The products and sums are rounded one by one (no contraction), and division
// and square root are IEEE, so the step gives the same bits as the formulas
// evaluated in that order in 32 bits.
//
// 8-bit states hold m and sqrt(v) in e4m3, 128 consecutive elements to a
// scale (the largest size over 448): sqrt(v) needs half of v's exponent
// range, and its three mantissa bits say as much as v's would.  p uses the
// new moments before they are rounded.  A decay of 0.999 changes v by less
// than half of an e4m3 step, so rounding to nearest can leave an element's
// code where it is for ever; with `stochastic` a moment goes up or down with
// the probabilities that keep its mean.  A second moment above zero keeps at
// least the smallest code: as zero it would divide m by eps alone.
#include "common.hpp"
#include "launch_train.hpp"
#include "train.hpp"

namespace fff {
namespace {

constexpr int kThreads = 256;
static_assert(kAdamwChunk == kThreads * 8 && kStateBlock == 16 * 8, "16 lanes hold a block");

// The entry whose workgroups `block` is one of (first ascending, e[0].first = 0).
template <typename Args>
__device__ __forceinline__ int entry_of(const Args& a, uint32_t block) {
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.e[mid].first <= block)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// MurmurHash3's 32-bit finaliser (Appleby; public domain).
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

// |t| <= 448 to an e4m3 value, down or up by the uniform u = bits / 2^16:
// floor(|t| / step + u) step, step = 2^(exponent - 3), at least 2^-9.
__device__ __forceinline__ float stochastic_e4m3(float t, uint32_t bits16) {
#pragma clang fp contract(off)
  const float a = fabsf(t);
  const uint32_t e = umax(__float_as_uint(a) >> 23, 121u);
  const float up = __uint_as_float((257u - e) << 23);
  const float down = __uint_as_float((e - 3u) << 23);
  const float k = floorf(a * up + static_cast<float>(bits16) * (1.0f / 65536.0f));
  return copysignf(fminf(k * down, kE4m3Max), t);
}

// 32 bits to bf16, up in size with the probability that the lost bits name.
__device__ __forceinline__ float stochastic_bf16(float v, uint32_t bits16) {
  const uint32_t b = __float_as_uint(v);
  if (size_bits(v) > 0x7f800000u) return v;  // NaN: the sum below could leave the format
  return __uint_as_float((b + bits16) & 0xffff0000u);
}

template <int PARAM, typename G, bool E4M3, bool STOCHASTIC>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
#pragma clang fp contract(off)
  const AdamwEntry& t = a.e[entry_of(a, blockIdx.x)];
  const int64_t i0 = int64_t(blockIdx.x - t.first) * kAdamwChunk + threadIdx.x * 8;
  const int n = t.n - i0 >= 8 ? 8 : static_cast<int>(t.n - i0 > 0 ? t.n - i0 : 0);
  using P = typename std::conditional<PARAM == kParamBf16, uint16_t, float>::type;
  P* const p = (PARAM == kParamMaster ? reinterpret_cast<P*>(t.master) : static_cast<P*>(t.param)) + i0;
  Eight<P> pr;
  Eight<G> gr;
  load_eight(pr, static_cast<const P*>(p), n);
  load_eight(gr, static_cast<const G*>(t.grad) + i0, n);
  float m[8], r[8];
  uint8_t* const mq = static_cast<uint8_t*>(t.exp_avg) + i0;
  uint8_t* const rq = static_cast<uint8_t*>(t.exp_avg_sq) + i0;
  float* const mf = static_cast<float*>(t.exp_avg) + i0;
  float* const vf = static_cast<float*>(t.exp_avg_sq) + i0;
  f32x2_t* const scale = reinterpret_cast<f32x2_t*>(t.scale) + i0 / kStateBlock;
  if constexpr (E4M3) {
    EightE4m3 qm, qr;
    qm.load(mq, n);
    qr.load(rq, n);
    f32x2_t sc = {0.0f, 0.0f};
    if (n > 0) sc = *scale;
    qm.get(m);
    qr.get(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] *= sc[0];
      r[i] *= sc[1];
      r[i] *= r[i];
    }
  } else {
    Eight<float> em, ev;
    load_eight(em, static_cast<const float*>(mf), n);
    load_eight(ev, static_cast<const float*>(vf), n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = em.get(i);
      r[i] = ev.get(i);
    }
  }
  float gs = 1.0f;
  if (a.grad_scale) gs = *a.grad_scale;
  float w[8];
  uint32_t top_m = 0, top_r = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = gr.get(i) * gs;
    m[i] = m[i] * a.beta1 + g * a.one_beta1;
    const float v = r[i] * a.beta2 + (g * g) * a.one_beta2;
    const float root = sqrtf(v);
    w[i] = pr.get(i) * t.decay - t.step * (m[i] / (root * a.root + a.eps));
    r[i] = E4M3 ? root : v;
    if (E4M3 && i < n) {
      top_m = umax(top_m, size_bits(m[i]));
      top_r = umax(top_r, size_bits(root));
    }
  }
  if (gs != gs) return;  // the gradient's norm was not finite: no step
  uint32_t h[8];
  if constexpr (STOCHASTIC) {
    const uint32_t base = t.key ^ (static_cast<uint32_t>(i0 >> 32) * 0x9E3779B9u);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = mix32((static_cast<uint32_t>(i0) + i) ^ base);
  }
  if constexpr (PARAM == kParamMaster) {
    store_eight(static_cast<uint16_t*>(t.param) + i0, n, w);
  } else if constexpr (PARAM == kParamBf16 && STOCHASTIC) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = stochastic_bf16(w[i], mix32(h[i] ^ 0x9E3779B9u) & 0xffffu);
    store_eight(p, n, v);
  }
  if constexpr (!(PARAM == kParamBf16 && STOCHASTIC)) store_eight(p, n, w);
  if constexpr (!E4M3) {
    store_eight(mf, n, m);
    store_eight(vf, n, r);
  } else {
    const float sm = e4m3_scale(group_max<16>(top_m));
    const float sr = e4m3_scale(group_max<16>(top_r));
    const float im = 1.0f / sm, ir = 1.0f / sr;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float tm = m[i] * im, tr = r[i] * ir;
      m[i] = STOCHASTIC ? stochastic_e4m3(tm, h[i] & 0xffffu) : tm;
      const float q = STOCHASTIC ? stochastic_e4m3(tr, h[i] >> 16) : tr;
      r[i] = tr > 0.0f ? fmaxf(q, 0.001953125f) : q;
    }
    if (n > 0) {
      store_e4m3(mq, n, m);
      store_e4m3(rq, n, r);
      if (threadIdx.x % 16 == 0) *scale = f32x2_t{sm, sr};
    }
  }
}

// Sum of squares of one chunk of one tensor, in 64 bits: neither a large
// gradient nor the number of elements costs the sum anything.
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(GradNormArgs a) {
  const GradEntry& t = a.e[entry_of(a, blockIdx.x)];
  const bool bf16 = t.n < 0;
  const int64_t n = bf16 ? -t.n : t.n;
  const int64_t begin = int64_t(blockIdx.x - t.first) * kNormChunk;
  double s = 0.0;
#pragma unroll 4
  for (int k = 0; k < kNormChunk / (kThreads * 8); ++k) {
    const int64_t i0 = begin + (k * kThreads + threadIdx.x) * 8;
    const int m = n - i0 >= 8 ? 8 : static_cast<int>(n - i0 > 0 ? n - i0 : 0);
    if (bf16) {
      Eight<uint16_t> g;
      load_eight(g, static_cast<const uint16_t*>(t.grad) + i0, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += static_cast<double>(g.get(i)) * g.get(i);
    } else {
      Eight<float> g;
      load_eight(g, static_cast<const float*>(t.grad) + i0, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += static_cast<double>(g.get(i)) * g.get(i);
    }
  }
  __shared__ double lds[kThreads / kWave];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, kWave);
  if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.partial[blockIdx.x] = lds[0] + lds[1] + lds[2] + lds[3];
}

__global__ __launch_bounds__(1024) void grad_norm_final_kernel(const double* partial, int64_t count,
                                                               double max_norm, float* out) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += 1024) s += partial[i];
  __shared__ double lds[16];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, kWave);
  if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < 16; ++i) s += lds[i];
    const float norm = static_cast<float>(sqrt(s));
    double factor = max_norm / (sqrt(s) + 1e-6);
    if (!(factor < 1.0)) factor = 1.0;
    out[0] = norm;
    out[1] = isfinite(norm) ? static_cast<float>(factor) : __uint_as_float(0x7fc00000u);
  }
}

template <int PARAM, typename G>
void launch_states(const AdamwArgs& a, int blocks, bool e4m3, bool stochastic, hipStream_t st) {
  if (e4m3 && stochastic)
    adamw_kernel<PARAM, G, true, true><<<blocks, kThreads, 0, st>>>(a);
  else if (e4m3)
    adamw_kernel<PARAM, G, true, false><<<blocks, kThreads, 0, st>>>(a);
  else if (stochastic && PARAM == kParamBf16)
    adamw_kernel<PARAM, G, false, PARAM == kParamBf16><<<blocks, kThreads, 0, st>>>(a);
  else  // nothing in this case is rounded stochastically
    adamw_kernel<PARAM, G, false, false><<<blocks, kThreads, 0, st>>>(a);
}

template <int PARAM>
void launch_grads(const AdamwArgs& a, int blocks, bool grad_bf16, bool e4m3, bool stochastic,
                  hipStream_t st) {
  if (grad_bf16)
    launch_states<PARAM, uint16_t>(a, blocks, e4m3, stochastic, st);
  else
    launch_states<PARAM, float>(a, blocks, e4m3, stochastic, st);
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, int blocks, int param, bool grad_bf16, bool state_e4m3,
                        bool stochastic, hipStream_t st) {
  if (param == kParamF32)
    launch_grads<kParamF32>(a, blocks, grad_bf16, state_e4m3, stochastic, st);
  else if (param == kParamBf16)
    launch_grads<kParamBf16>(a, blocks, grad_bf16, state_e4m3, stochastic, st);
  else
    launch_grads<kParamMaster>(a, blocks, grad_bf16, state_e4m3, stochastic, st);
  return hipGetLastError();
}

hipError_t launch_grad_squares(const GradNormArgs& a, int blocks, hipStream_t st) {
  grad_squares_kernel<<<blocks, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_norm_final(const double* partial, int64_t count, double max_norm, float* out,
                                  hipStream_t st) {
  grad_norm_final_kernel<<<1, 1024, 0, st>>>(partial, count, max_norm, out);
  return hipGetLastError();
}

}  // namespace fff
