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

constexpr uint32_t kFirstMask = (1u << kFirstBits) - 1;

// The entry whose workgroups `block` is one of: the last whose first
// workgroup (the low 24 bits of first[], ascending from 0) is not past it.
// Each lane looks at its own entries, so the search costs one load and not a
// chain of them.
template <int MOST>
__device__ __forceinline__ int entry_of(const uint32_t (&first)[MOST], int count, uint32_t block) {
  int at = -1;
#pragma unroll
  for (int base = 0; base < MOST; base += kWave) {
    const int i = base + (threadIdx.x & (kWave - 1));
    at += __popcll(__ballot(i < count && (first[i < MOST ? i : 0] & kFirstMask) <= block));
  }
  return at;
}

// MurmurHash3's 32-bit finaliser (Appleby; public domain).
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

// Eight elements from i0 on; n of them (8 where FULL) belong to the tensor.
template <int PARAM, typename G, bool E4M3, bool STOCHASTIC, bool FULL>
__device__ __forceinline__ void adamw_eight(const AdamwArgs& a, const AdamwEntry& t, int64_t size,
                                            int64_t i0) {
#pragma clang fp contract(off)
  const int n = FULL || size - i0 >= 8 ? 8 : static_cast<int>(size - i0 > 0 ? size - i0 : 0);
  using P = typename std::conditional<PARAM == kParamBf16, uint16_t, float>::type;
  P* const p = t.get<P>(PARAM == kParamMaster ? t.kMaster : t.kParam) + i0;
  Eight<P> pr;
  Eight<G> gr;
  load_eight(pr, static_cast<const P*>(p), n);
  load_eight(gr, t.get<const G>(t.kGrad) + i0, n);
  float m[8], r[8];
  uint8_t* const mq = t.get<uint8_t>(t.kExpAvg) + i0;
  uint8_t* const rq = t.get<uint8_t>(t.kExpAvgSq) + i0;
  float* const mf = t.get<float>(t.kExpAvg) + i0;
  float* const vf = t.get<float>(t.kExpAvgSq) + i0;
  f32x2_t* const scale = t.get<f32x2_t>(t.kScale) + i0 / kStateBlock;
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
    if (E4M3) {
      top_m = umax(top_m, size_bits(m[i]));
      top_r = umax(top_r, __float_as_uint(root));  // root >= 0, or NaN
    }
  }
  if (gs != gs) return;  // the gradient's norm was not finite: no step
  uint32_t h[8], rnd[8];
  if constexpr (STOCHASTIC) {
    const uint32_t base = t.key ^ (static_cast<uint32_t>(i0 >> 32) * 0x9E3779B9u);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = mix32((static_cast<uint32_t>(i0) + i) ^ base);
  }
  if constexpr (PARAM == kParamMaster) store_eight(t.get<uint16_t>(t.kParam) + i0, n, w);
  if constexpr (PARAM == kParamBf16 && STOCHASTIC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rnd[i] = mix32(h[i] ^ 0x9E3779B9u) << 16;
    store_packed(p, n, pack_bf16_stochastic(w, rnd));
  } else {
    store_eight(p, n, w);
  }
  if constexpr (!E4M3) {
    store_eight(mf, n, m);
    store_eight(vf, n, r);
    return;
  }
  // Lanes past the tensor's end hold zeros, which no maximum sees.
  const float sm = e4m3_scale(group_max<16>(top_m));
  const float sr = e4m3_scale(group_max<16>(top_r));
  const float im = 1.0f / sm, ir = 1.0f / sr;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] *= im;
    r[i] *= ir;
    // at least the smallest code, which every rounding of it keeps
    r[i] = r[i] > 0.0f ? fmaxf(r[i], 0.001953125f) : r[i];
  }
  u32x2_t qm, qr;
  if constexpr (STOCHASTIC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rnd[i] = h[i] << 16;
    qm = pack_e4m3_stochastic(m, rnd);
#pragma unroll
    for (int i = 0; i < 8; ++i) rnd[i] = h[i] & 0xffff0000u;
    qr = pack_e4m3_stochastic(r, rnd);
  } else {
    qm = pack_e4m3(m);
    qr = pack_e4m3(r);
  }
  if (n > 0) {
    store_packed(mq, n, qm);
    store_packed(rq, n, qr);
    if (threadIdx.x % 16 == 0) *scale = f32x2_t{sm, sr};
  }
}

// One chunk of one tensor.  A chunk inside its tensor runs without any tests
// for the tensor's end.
template <int PARAM, typename G, bool E4M3, bool STOCHASTIC>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
  const int at = entry_of(a.first, a.count, blockIdx.x);
  const AdamwEntry& t = a.e[at];
  const uint32_t first = a.first[at];
  const int64_t size = int64_t(first >> kFirstBits) << 32 | t.n_lo;
  const int64_t begin = int64_t(blockIdx.x - (first & kFirstMask)) * kAdamwChunk;
  if (size - begin >= kAdamwChunk)
    adamw_eight<PARAM, G, E4M3, STOCHASTIC, true>(a, t, size, begin + threadIdx.x * 8);
  else
    adamw_eight<PARAM, G, E4M3, STOCHASTIC, false>(a, t, size, begin + threadIdx.x * 8);
}

// Sum of squares of one chunk of one tensor, in 64 bits: neither a large
// gradient nor the number of elements costs the sum anything.
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(GradNormArgs a) {
  const int at = entry_of(a.first, a.count, blockIdx.x);
  const GradEntry& t = a.e[at];
  const bool bf16 = t.n < 0;
  const int64_t n = bf16 ? -t.n : t.n;
  const int64_t begin = int64_t(blockIdx.x - a.first[at]) * kNormChunk;
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
