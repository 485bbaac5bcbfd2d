// AdamW over many tensors in one launch, with moments in 32 or in 8 bits, and
// the gradient's norm over many tensors.
//
// Per element, with g already times *grad_scale:
//   m = m beta1 + g (1 - beta1);   v = v beta2 + (g g) (1 - beta2)
//   p = p decay - step (m / (sqrt(v) root + eps))
// with decay = 1 - lr wd, step = lr / (1 - beta1^t) and root = 1 / sqrt(1 - beta2^t)
// from the host, formed in 64 bits and rounded to 32.
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
//
// Bound by HBM with 32-bit states: 17.2 M weights with masters, 30 bytes each,
// take 86.9 us (6.0 TB/s; a large copy reaches 5.3).  With 8-bit states the
// vector ALU comes close: 18.2 bytes a weight with masters take 54.3 us (5.8
// TB/s, ALU 53 % busy), 12.1 without, all rounded stochastically, 44.8 us for
// 19.5 M (5.3 TB/s, 82 % busy).  A workgroup has 2048 elements, a lane two
// quads of four: as many loads in flight as a kernel of one pass needs, and
// 16-byte accesses that are contiguous over the wavefront (eight consecutive
// elements a lane read at the same rate, but streaming accesses then lose:
// 120 us instead of 89 in a model of the step).
#include "common.hpp"
#include "launch_train.hpp"
#include "train.hpp"

namespace fff {
namespace {

constexpr int kThreads = 256;
constexpr int kV = 4;  // consecutive elements of a lane: 16 bytes in 32 bits
constexpr int kQuads = kAdamwChunk / (kThreads * kV);
static_assert(kStateBlock == 32 * kV, "32 lanes hold a block");

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

// What a lane has of one quad: its elements, as loaded and then as updated.
template <typename P, typename G, bool E4M3>
struct Quad {
  using State = typename std::conditional<E4M3, uint8_t, float>::type;
  int64_t i0;
  int n;  // of its four elements, how many the tensor has
  Pack<P, kV> p;
  Pack<G, kV> g;
  Pack<State, kV> m, v;
  f32x2_t scale;
};

// Correctly rounded square root and quotient by an approximation, its error
// by fma and one correction (Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990): 36 cycles of a wavefront
// each where the compiler's, which also serve operands near the ends of the
// range, take 76 and 52; the 8-bit step is bound by them.  The root is the
// IEEE one for v = 0 and every v in [2^-90, 2^60) (the tests compare all of
// them).  The quotient is for m = 0 and m in [2^-60, 2^60) over [2^-60, 2^90):
// no pair of 1e11 differed, every mantissa of m over 12288 divisors, the 4096
// smallest and the 4096 largest mantissas among them.  That is a sample of
// the divisors; the tests hold 48 of them.
__device__ __forceinline__ float short_sqrt(float v) {
#pragma clang fp contract(off)
  const float y = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-126f));  // (finite for v = 0)
  const float g = v * y;
  return __builtin_fmaf(__builtin_fmaf(-g, g, v), 0.5f * y, g);
}

__device__ __forceinline__ float short_div(float m, float d) {
#pragma clang fp contract(off)
  float y = __builtin_amdgcn_rcpf(d);
  y = __builtin_fmaf(__builtin_fmaf(-d, y, 1.0f), y, y);
  const float q = m * y;
  return __builtin_fmaf(__builtin_fmaf(-q, d, m), y, q);
}

// The ranges' ends as bits(v) - 1 (zero wraps to the top) and bits(v); m's
// lower end is in AdamwArgs::long_m.
constexpr uint32_t kShortLowV = (37u << 23) - 1;  // 2^-90
constexpr uint32_t kShortTopV = 187u << 23;       // 2^60
constexpr float kShortTop = 0x1p60f;

__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// One chunk of one tensor (FULL: all of it inside the tensor, which then
// needs no tests for the end).  A lane's quads are kThreads * kV apart, so
// that every access of a wavefront is contiguous; all are loaded before the
// first is used.
template <int PARAM, typename G, bool E4M3, bool STOCHASTIC, bool STREAM, bool FULL>
__device__ __forceinline__ void adamw_chunk(const AdamwArgs& a, const AdamwEntry& t, int64_t size,
                                            int64_t begin) {
#pragma clang fp contract(off)
  using P = typename std::conditional<PARAM == kParamBf16, uint16_t, float>::type;
  using Q = Quad<P, G, E4M3>;
  using State = typename Q::State;
  P* const p = t.get<P>(PARAM == kParamMaster ? t.kMaster : t.kParam);
  const G* const grad = t.get<const G>(t.kGrad);
  State* const ms = t.get<State>(t.kExpAvg);
  State* const vs = t.get<State>(t.kExpAvgSq);
  float* const scales = t.get<float>(t.kScale);
  Q q[kQuads];
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    q[k].i0 = begin + (k * kThreads + threadIdx.x) * kV;
    const int64_t left = size - q[k].i0;
    const int n = q[k].n = FULL || left >= kV ? kV : static_cast<int>(left > 0 ? left : 0);
    q[k].p.template load<STREAM>(p + q[k].i0, n);
    q[k].g.template load<STREAM>(grad + q[k].i0, n);
    q[k].m.template load<STREAM>(ms + q[k].i0, n);
    q[k].v.template load<STREAM>(vs + q[k].i0, n);
    q[k].scale = f32x2_t{0.0f, 0.0f};
    if (E4M3 && n > 0)
      q[k].scale = *reinterpret_cast<const f32x2_t*>(scales + q[k].i0 / kStateBlock * 2);
  }
  float gs = 1.0f;
  if (a.grad_scale) gs = *a.grad_scale;
  if (gs != gs) return;  // the gradient's norm was not finite: no step
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int64_t i0 = q[k].i0;
    const int n = q[k].n;
    float m[kV], r[kV], w[kV];
    if constexpr (E4M3) {
      unpack_e4m3(q[k].m, m);
      unpack_e4m3(q[k].v, r);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        m[i] *= q[k].scale[0];
        r[i] *= q[k].scale[1];
        r[i] *= r[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        m[i] = q[k].m.get(i);
        r[i] = q[k].v.get(i);
      }
    }
    // m / denominator and sqrt(v) in the short forms where every operand of
    // this lane is zero or in their range, which is all but always.
    float v[kV], ratio[kV];
    uint32_t low_m = ~0u, low_v = ~0u;  // smallest sizes above zero, zero as the largest
    uint32_t top_v = 0;  // as bits: NaN and anything below zero are above every number
    float top_m = 0.0f, top_r = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const float g = q[k].g.get(i) * gs;
      m[i] = m[i] * a.beta1 + g * a.one_beta1;
      v[i] = r[i] * a.beta2 + (g * g) * a.one_beta2;
      r[i] = short_sqrt(v[i]);
      ratio[i] = short_div(m[i], r[i] * a.root + a.eps);
      low_m = umin(low_m, 2 * __float_as_uint(m[i]) - 1);
      low_v = umin(low_v, __float_as_uint(v[i]) - 1);
      top_m = fmaxf(top_m, fabsf(m[i]));
      top_r = fmaxf(top_r, r[i]);
      top_v = umax(top_v, __float_as_uint(v[i]));
    }
    if (low_m <= a.long_m || low_v < kShortLowV || !(top_m < kShortTop) || top_v >= kShortTopV) {
      top_r = 0.0f;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        r[i] = sqrtf(v[i]);
        ratio[i] = m[i] / (r[i] * a.root + a.eps);
        top_r = fmaxf(top_r, r[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) w[i] = q[k].p.get(i) * t.decay - t.step * ratio[i];
    uint32_t h[kV], rnd[kV];
    if constexpr (STOCHASTIC) {
      const uint32_t base = t.key ^ (static_cast<uint32_t>(i0 >> 32) * 0x9E3779B9u);
#pragma unroll
      for (int i = 0; i < kV; ++i) h[i] = mix32((static_cast<uint32_t>(i0) + i) ^ base);
    }
    if constexpr (PARAM == kParamMaster)
      packed<uint16_t, kV>(w).template store<STREAM>(t.get<uint16_t>(t.kParam) + i0, n);
    if constexpr (PARAM == kParamBf16 && STOCHASTIC) {
#pragma unroll
      for (int i = 0; i < kV; ++i) rnd[i] = mix32(h[i] ^ 0x9E3779B9u) << 16;
      pack_bf16_stochastic(w, rnd).template store<STREAM>(p + i0, n);
    } else {
      packed<P, kV>(w).template store<STREAM>(p + i0, n);
    }
    if constexpr (!E4M3) {
      packed<float, kV>(m).template store<STREAM>(ms + i0, n);
      packed<float, kV>(v).template store<STREAM>(vs + i0, n);
      continue;
    }
    // The block's 32 lanes are two rows of 16.  One swap of the rows leaves
    // both maxima of m in the first row and both of r in the second, so that
    // one division serves both scales; another gives every lane both.
    // Lanes past the tensor's end hold zeros, which no maximum sees.
    const auto top = __builtin_amdgcn_permlane16_swap(
        group_max<16>(__float_as_uint(top_m)), group_max<16>(__float_as_uint(top_r)), false, false);
    const float scale = e4m3_scale(umax(top[0], top[1]));
    const float inv = reciprocal(scale);
    const auto both = __builtin_amdgcn_permlane16_swap(__float_as_uint(inv), __float_as_uint(inv),
                                                       false, false);
    const float im = __uint_as_float(both[0]), ir = __uint_as_float(both[1]);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      m[i] *= im;
      r[i] *= ir;
      // above zero, at least the smallest code, which every rounding keeps
      r[i] = r[i] > 0.0f ? fmaxf(r[i], 0x1p-9f) : r[i];
    }
    Pack<uint8_t, kV> qm, qr;
    if constexpr (STOCHASTIC) {
#pragma unroll
      for (int i = 0; i < kV; ++i) rnd[i] = h[i] << 16;
      qm = pack_e4m3_stochastic(m, rnd);
#pragma unroll
      for (int i = 0; i < kV; ++i) rnd[i] = h[i] & 0xffff0000u;
      qr = pack_e4m3_stochastic(r, rnd);
    } else {
      qm = pack_e4m3(m);
      qr = pack_e4m3(r);
    }
    if constexpr (E4M3) {
      qm.template store<STREAM>(ms + i0, n);
      qr.template store<STREAM>(vs + i0, n);
      // the first lane of either row; the block's first element is in the first one
      const int64_t block = i0 / kStateBlock;
      if (threadIdx.x % 16 == 0 && block * kStateBlock < size)
        scales[2 * block + (threadIdx.x / 16) % 2] = scale;
    }
  }
}

template <int PARAM, typename G, bool E4M3, bool STOCHASTIC, bool STREAM>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
  const int at = entry_of(a.first, a.count, blockIdx.x);
  const AdamwEntry& t = a.e[at];
  const uint32_t first = a.first[at];
  const int64_t size = int64_t(first >> kFirstBits) << 32 | t.n_lo;
  const int64_t begin = int64_t(blockIdx.x - (first & kFirstMask)) * kAdamwChunk;
  if (size - begin >= kAdamwChunk)
    adamw_chunk<PARAM, G, E4M3, STOCHASTIC, STREAM, true>(a, t, size, begin);
  else
    adamw_chunk<PARAM, G, E4M3, STOCHASTIC, STREAM, false>(a, t, size, begin);
}

// A lane's share of the squares of one chunk of CHUNK elements of a tensor,
// 16 bytes at a time, by LANES lanes.
template <typename E, int CHUNK, int LANES, bool STREAM>
__device__ __forceinline__ double squares(const E* grad, int64_t n, int64_t begin, int lane) {
  constexpr int V = 16 / int(sizeof(E));
  double s = 0.0;
#pragma unroll 8
  for (int k = 0; k < CHUNK / (LANES * V); ++k) {
    const int64_t i0 = begin + (k * LANES + lane) * V;
    Pack<E, V> g;
    g.template load<STREAM>(grad + i0, n - i0 >= V ? V : static_cast<int>(n - i0 > 0 ? n - i0 : 0));
#pragma unroll
    for (int i = 0; i < V; ++i) s += static_cast<double>(g.get(i)) * g.get(i);
  }
  return s;
}

// Chunk `chunk` of the list.  Squares are added in 64 bits: neither a large
// gradient nor the number of elements costs the sum anything, and the
// additions hide behind the loads.
template <int CHUNK, int LANES, bool STREAM>
__device__ __forceinline__ double chunk_squares(const GradNormArgs& a, uint32_t chunk, int lane) {
  const int at = entry_of(a.first, a.count, chunk);
  const GradEntry& t = a.e[at];
  const int64_t begin = int64_t(chunk - (a.first[at] & kFirstMask)) * CHUNK;
  if (t.n < 0)
    return squares<uint16_t, CHUNK, LANES, STREAM>(static_cast<const uint16_t*>(t.grad), -t.n, begin,
                                                   lane);
  return squares<float, CHUNK, LANES, STREAM>(static_cast<const float*>(t.grad), t.n, begin, lane);
}

// Sum over the workgroup, added in one order; thread 0 gets it.
template <int THREADS>
__device__ __forceinline__ double block_total(double s) {
  __shared__ double lds[THREADS / kWave];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, kWave);
  if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = s;
  __syncthreads();
  s = 0.0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) s += lds[i];
  }
  return s;
}

__device__ __forceinline__ void write_norm(double squares, double max_norm, float* out) {
  const double root = sqrt(squares);
  const float norm = static_cast<float>(root);
  double factor = max_norm / (root + 1e-6);
  if (!(factor < 1.0)) factor = 1.0;
  out[0] = norm;
  out[1] = isfinite(norm) ? static_cast<float>(factor) : __uint_as_float(0x7fc00000u);
}

template <bool STREAM>
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(GradNormArgs a) {
  const double s = block_total<kThreads>(
      chunk_squares<kNormChunk, kThreads, STREAM>(a, blockIdx.x, threadIdx.x));
  if (threadIdx.x == 0) a.partial[blockIdx.x] = s;
}

// The sum of the partials, in one order.  A second launch: with a count of
// the workgroups that are done, by which the last one would do this itself,
// 1054 atomics on one address made 24 us of 14.
__global__ __launch_bounds__(1024) void grad_norm_final_kernel(const double* partial, int64_t count,
                                                               double max_norm, float* out) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += 1024) s += partial[i];
  s = block_total<1024>(s);
  if (threadIdx.x == 0) write_norm(s, max_norm, out);
}

// All of a small list (128 K elements) in one workgroup, a chunk per wavefront
// at a time: one launch and no workspace, 7.8 us a call for 96 K elements
// where the two launches take 9.8; 172 K would take 11.9 and 9.6.
__global__ __launch_bounds__(1024) void grad_norm_small_kernel(GradNormArgs a, uint32_t chunks,
                                                               double max_norm, float* out) {
  double s = 0.0;
  for (uint32_t c = threadIdx.x / kWave; c < chunks; c += 1024 / kWave)
    s += chunk_squares<kNormSmallChunk, kWave, false>(a, c, threadIdx.x % kWave);
  s = block_total<1024>(s);
  if (threadIdx.x == 0) write_norm(s, max_norm, out);
}

template <int PARAM, typename G, bool STREAM>
void launch_states(const AdamwArgs& a, int blocks, bool e4m3, bool stochastic, hipStream_t st) {
  if (e4m3 && stochastic)
    adamw_kernel<PARAM, G, true, true, STREAM><<<blocks, kThreads, 0, st>>>(a);
  else if (e4m3)
    adamw_kernel<PARAM, G, true, false, STREAM><<<blocks, kThreads, 0, st>>>(a);
  else if (stochastic && PARAM == kParamBf16)
    adamw_kernel<PARAM, G, false, PARAM == kParamBf16, STREAM><<<blocks, kThreads, 0, st>>>(a);
  else  // nothing in this case is rounded stochastically
    adamw_kernel<PARAM, G, false, false, STREAM><<<blocks, kThreads, 0, st>>>(a);
}

template <int PARAM, bool STREAM>
void launch_grads(const AdamwArgs& a, int blocks, bool grad_bf16, bool e4m3, bool stochastic,
                  hipStream_t st) {
  if (grad_bf16)
    launch_states<PARAM, uint16_t, STREAM>(a, blocks, e4m3, stochastic, st);
  else
    launch_states<PARAM, float, STREAM>(a, blocks, e4m3, stochastic, st);
}

template <bool STREAM>
void launch_params(const AdamwArgs& a, int blocks, int param, bool grad_bf16, bool e4m3,
                   bool stochastic, hipStream_t st) {
  if (param == kParamF32)
    launch_grads<kParamF32, STREAM>(a, blocks, grad_bf16, e4m3, stochastic, st);
  else if (param == kParamBf16)
    launch_grads<kParamBf16, STREAM>(a, blocks, grad_bf16, e4m3, stochastic, st);
  else
    launch_grads<kParamMaster, STREAM>(a, blocks, grad_bf16, e4m3, stochastic, st);
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, int blocks, int param, bool grad_bf16, bool state_e4m3,
                        bool stochastic, hipStream_t st) {
  if (adamw_streams(blocks, param, grad_bf16, state_e4m3))
    launch_params<true>(a, blocks, param, grad_bf16, state_e4m3, stochastic, st);
  else
    launch_params<false>(a, blocks, param, grad_bf16, state_e4m3, stochastic, st);
  return hipGetLastError();
}

// 275 MB of gradients take 46.8 us past the caches and 52.0 through them.
// Fewer bytes stay in the last-level cache for the step that reads them next.
hipError_t launch_grad_squares(const GradNormArgs& a, int blocks, hipStream_t st) {
  int64_t bytes = 0;
  for (int i = 0; i < a.count; ++i) bytes += a.e[i].n < 0 ? -2 * a.e[i].n : 4 * a.e[i].n;
  if (bytes >= kStreamBytes)
    grad_squares_kernel<true><<<blocks, kThreads, 0, st>>>(a);
  else
    grad_squares_kernel<false><<<blocks, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_norm_small(const GradNormArgs& a, uint32_t chunks, double max_norm, float* out,
                                  hipStream_t st) {
  grad_norm_small_kernel<<<1, 1024, 0, st>>>(a, chunks, max_norm, out);
  return hipGetLastError();
}

hipError_t launch_grad_norm_final(const double* partial, int64_t count, double max_norm, float* out,
                                  hipStream_t st) {
  grad_norm_final_kernel<<<1, 1024, 0, st>>>(partial, count, max_norm, out);
  return hipGetLastError();
}

}  // namespace fff
