// Device code shared by the dense feed-forward kernels: activations and their
// slopes, values kept for the backward pass, and the epilogues of the
// products.
#pragma once

#include "common.hpp"
#include "launch_dense.hpp"
#include "mfma_tile.hpp"
#include "train.hpp"

namespace fff {

// fff_act_t
enum { kActNone = 0, kActGelu = 1, kActSilu = 2, kActRelu = 3 };

// Lanes of one scale's group, four (or V) columns a lane.
template <int V>
__device__ __forceinline__ uint32_t scale_group_top(uint32_t v, int group) {
  if (group == 32) return group_max<32 / V>(v);
  if (group == 64) return group_max<64 / V>(v);
  return group_max<128 / V>(v);
}

// The logistic function 1 / (1 + exp(-z)).  exp2's argument is rounded once,
// so the result is off by about (|z| + 3) 2^-24 of itself.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// GELU in its tanh form is a times the logistic function of
// 2 sqrt(2/pi) (a + 0.044715 a^3); SiLU a times that of a.
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGelu3 = 0.044715f;

__device__ __forceinline__ float activation(float a, int act) {
  switch (act) {
    case kActGelu: return a * logistic(kGelu2 * (a + kGelu3 * (a * a * a)));
    case kActSilu: return a * logistic(a);
    case kActRelu: return a < 0.0f ? 0.0f : a;  // (NaN stays)
    default: return a;
  }
}

// The activation and its derivative.
__device__ __forceinline__ void activation_slope(float a, int act, float& value, float& slope) {
  switch (act) {
    // (where q is 0 or 1 the second term is nothing, but its factors may be
    // infinite: values beyond 1e19, infinities)
    case kActGelu: {
      const float q = logistic(kGelu2 * (a + kGelu3 * (a * a * a)));
      value = a * q;
      const float more = value * (1.0f - q) * (kGelu2 * (1.0f + 3.0f * kGelu3 * (a * a)));
      slope = q * (1.0f - q) == 0.0f ? q : q + more;
      break;
    }
    case kActSilu: {
      const float q = logistic(a);
      value = a * q;
      slope = q * (1.0f - q) == 0.0f ? q : q + value * (1.0f - q);
      break;
    }
    case kActRelu:
      value = a < 0.0f ? 0.0f : a;
      slope = a > 0.0f ? 1.0f : (a <= 0.0f ? 0.0f : a);
      break;
    default:
      value = a;
      slope = 1.0f;
  }
}

// V consecutive columns of a row, n of them there, into 8 bits with the scale
// of their group of 32, 64 or 128 columns: every lane of the group takes
// part, in columns 0, V, 2V, ... of the row.
template <int V>
__device__ __forceinline__ void save_e4m3(const float (&v)[V], int n, uint8_t* codes, float* scales,
                                          int64_t row, int col, int N, int group) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) top = umax(top, i < n ? size_bits(v[i]) : 0u);
  top = scale_group_top<V>(top, group);
  const float scale = e4m3_scale(top);
  const float inv = reciprocal(scale);
  float q[V];
#pragma unroll
  for (int i = 0; i < V; ++i) q[i] = v[i] * inv;
  if (n <= 0) return;
  pack_e4m3(q).store(codes + static_cast<size_t>(row) * N + col, n);
  if (col % group == 0)
    scales[static_cast<size_t>(row) * ((N + group - 1) / group) + col / group] = scale;
}

// V values into three planes, the first n of them stored; whether one is
// beyond the planes.  high is the nearest bf16, middle and low what is left,
// to nearest: high + middle + low is the value where low is above bf16's
// smallest (values above 2^-110), and off by at most 2^-134 below.
//
// Beyond are values that are not finite (infinity times a plane's zero would
// be NaN) and those of 2^47 or more: with smaller ones every sum of the at
// most 2^31 products stays below 2^125, whatever the terms' order and the
// middle and low parts' signs.  With larger ones a sum that float32 has as
// infinity could be infinity minus infinity.
constexpr float kPlanesEnd = 0x1p47f;
template <int V>
__device__ __forceinline__ bool store_planes(const float (&v)[V], uint16_t* at, int64_t plane, int n) {
  float part[3][V];
  bool odd = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    odd |= size_bits(v[i]) >= __float_as_uint(kPlanesEnd);
    const float h = bf16_to_f32(f32_to_bf16(v[i]));
    const float r = v[i] - h;
    const float m = bf16_to_f32(f32_to_bf16(r));
    part[0][i] = h;
    part[1][i] = m;
    part[2][i] = r - m;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) packed<uint16_t, V>(part[k]).store(at + k * plane, n);
  return odd;
}

// Epilogues.  apply() has four consecutive columns of a row, n (0 to 4) of
// them there; lanes of 128 aligned columns come together, so that the groups
// of 8-bit saves are complete.
template <typename E>
__device__ __forceinline__ void save_sums(const Epilogue& e, int which, int64_t row, int col, int n,
                                          const float (&v)[4]) {
  if (!e.save[which]) return;
  if (e.scale[which]) {
    save_e4m3(v, n, static_cast<uint8_t*>(e.save[which]), e.scale[which], row, col, e.N, e.group);
  } else if (n > 0) {
    packed<E, 4>(v).store(static_cast<E*>(e.save[which]) + static_cast<size_t>(row) * e.N + col, n);
  }
}

// out = act(v + bias) + residual: E the layer's type, O that of out and residual.
template <typename E, typename O>
struct LinearEpilogue {
  static constexpr bool kGated = false;
  Epilogue e;
  struct Column {
    float bias[4];
  };
  struct Early {
    Pack<O, 4> r;
  };
  __device__ __forceinline__ void column(Column& c, int col) const {
    Pack<E, 4> b = {};
    if (e.bias) b.load(static_cast<const E*>(e.bias) + col, e.N - col);
#pragma unroll
    for (int i = 0; i < 4; ++i) c.bias[i] = b.get(i);
  }
  // What an apply() reads, asked for ahead of it.
  __device__ __forceinline__ void early(Early& x, int64_t row, int col, int n) const {
    if (e.residual)
      x.r.load(static_cast<const O*>(e.residual) + static_cast<size_t>(row) * e.N + col, n);
  }
  __device__ __forceinline__ void apply(const Column& c, const Early& x, int64_t row, int col, int n,
                                        const float (&v)[4], const float (&)[4], int which) const {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = v[i] + c.bias[i];
    save_sums<E>(e, 0, row, col, n, y);
    if (n <= 0) return;
    if (e.act != kActNone) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = activation(y[i], e.act);
    }
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += x.r.get(i);
    }
    packed<O, 4>(y).store(static_cast<O*>(e.out[which]) + static_cast<size_t>(row) * e.N + col, n);
  }
};

// out = act(v) * w.
template <typename E>
struct GatedEpilogue {
  static constexpr bool kGated = true;
  Epilogue e;
  struct Column {};
  struct Early {};
  __device__ __forceinline__ void column(Column&, int) const {}
  __device__ __forceinline__ void early(Early&, int64_t, int, int) const {}
  __device__ __forceinline__ void apply(const Column&, const Early&, int64_t row, int col, int n,
                                        const float (&v)[4], const float (&w)[4], int) const {
    save_sums<E>(e, 0, row, col, n, v);
    save_sums<E>(e, 1, row, col, n, w);
    if (n <= 0) return;
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = activation(v[i], e.act) * w[i];
    packed<E, 4>(y).store(static_cast<E*>(e.out[0]) + static_cast<size_t>(row) * e.N + col, n);
  }
};

// Partial sums of one slice of K: [slice][v, w][M][N] in 32 bits.
template <bool GATED>
struct PartialEpilogue {
  static constexpr bool kGated = GATED;
  float* partial;
  int64_t M;
  int N;
  int products;  // sums of a slice: two of kPairColumns and kPairTwo
  struct Column {};
  struct Early {};
  __device__ __forceinline__ void column(Column&, int) const {}
  __device__ __forceinline__ void early(Early&, int64_t, int, int) const {}
  __device__ __forceinline__ void apply(const Column&, const Early&, int64_t row, int col, int n,
                                        const float (&v)[4], const float (&w)[4], int which) const {
    if (n <= 0) return;
    float* p = partial + (static_cast<size_t>(which) * M + row) * N + col;
    packed<float, 4>(v).store(p, n);
    if constexpr (GATED) packed<float, 4>(w).store(p + static_cast<size_t>(M) * N, n);
  }
  __device__ __forceinline__ void slice(int s) {
    partial += static_cast<size_t>(s) * products * M * N;
  }
};

// Accumulators of a tile (the layout of mma_frags) through LDS to an
// epilogue, a band of 32 rows of every wavefront row at a time, so that the
// lanes of a wavefront have consecutive columns: residuals are read and
// outputs written in whole lines, and an 8-bit save's groups are at hand.
// GATED: the first half of a wavefront's column blocks is of v, the second
// of w.
template <class C>
constexpr int band_pitch() { return C::BN + 4; }  // floats
template <class C>
constexpr size_t band_bytes() { return size_t(C::kWavesM) * 32 * band_pitch<C>() * sizeof(float); }

template <class C, class Epi>
__device__ __forceinline__ void tile_epilogue(const f32x16_t (&acc)[C::kTm][C::kTn],
                                              unsigned char* lds, const Epi& epi, int64_t m0,
                                              int64_t M, int n0, int N, int which) {
  constexpr bool G = Epi::kGated;
  constexpr int kPitch = band_pitch<C>();
  constexpr int kCols = G ? C::BN / 2 : C::BN;  // output columns of the tile
  constexpr int kRowsAtOnce = C::kThreads * 4 / kCols;
  constexpr int kRounds = 4;  // at a time
  constexpr int kBandRows = C::kWavesM * 32;
  static_assert(kCols >= 128 && kBandRows % (kRowsAtOnce * kRounds) == 0, "bands in whole rounds");
  float* band = reinterpret_cast<float*>(lds);
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = tid / kWave;
  const int wm = wave / C::kWavesN;
  const int wn = wave % C::kWavesN;
  const int c4 = (tid % (kCols / 4)) * 4;
  const int col = n0 + c4;
  typename Epi::Column column;
  epi.column(column, col);
  const int left = N - col;
  const int n_col = left < 0 ? 0 : left < 4 ? left : 4;
#pragma unroll
  for (int i = 0; i < C::kTm; ++i) {
    __syncthreads();  // the stages, or the previous band, have been read
#pragma unroll
    for (int j = 0; j < C::kTn; ++j) {
      const int cj = G ? j / (C::kTn / 2) * (C::BN / 2) + wn * (C::WN / 2) + j % (C::kTn / 2) * 32
                       : wn * C::WN + j * 32;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(band + (wm * 32 + (lane & 31)) * kPitch + cj + g * 8 +
                                   (lane >> 5) * 4) =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                        acc[i][j][4 * g + 3]);
    }
    __syncthreads();
    for (int u0 = 0; u0 < kBandRows; u0 += kRowsAtOnce * kRounds) {
      typename Epi::Early early[kRounds];
      auto row_of = [&](int u) {
        const int b = tid / (kCols / 4) + u0 + u * kRowsAtOnce;
        return m0 + (b / 32) * C::WM + i * 32 + b % 32;
      };
#pragma unroll
      for (int u = 0; u < kRounds; ++u)
        epi.early(early[u], row_of(u), col, row_of(u) < M ? n_col : 0);
#pragma unroll
      for (int u = 0; u < kRounds; ++u) {
        const int b = tid / (kCols / 4) + u0 + u * kRowsAtOnce;
        const float4 p = *reinterpret_cast<const float4*>(band + b * kPitch + c4);
        const float v[4] = {p.x, p.y, p.z, p.w};
        float w[4] = {};
        if constexpr (G) {
          const float4 q = *reinterpret_cast<const float4*>(band + b * kPitch + C::BN / 2 + c4);
          w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
        }
        epi.apply(column, early[u], row_of(u), col, row_of(u) < M ? n_col : 0, v, w, which);
      }
    }
  }
}

// Which tile, slice of K and product a workgroup has.  Tiles go in groups of
// eight row panels, rows first, so that the workgroups an XCD runs together
// share operand panels in its L2.
struct TileAt {
  int tm, tn, slice, which;
};
__device__ __forceinline__ TileAt tile_at(int tiles_m, int tiles_n, int products) {
  const int per = tiles_m * tiles_n;
  int t = xcd_logical_tile(blockIdx.x, gridDim.x);
  TileAt at;
  at.which = (t / per) % products;
  at.slice = t / per / products;
  t %= per;
  const int group = t / (8 * tiles_n);
  const int first = group * 8;
  const int rows = tiles_m - first < 8 ? tiles_m - first : 8;
  const int in = t - group * 8 * tiles_n;
  at.tm = first + in % rows;
  at.tn = in / rows;
  return at;
}

}  // namespace fff
