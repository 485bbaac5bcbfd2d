// Root-mean-square norm of rows with the residual's addition, its output in
// the layer's type or in e4m3 with scales:
//
//   z = x + r;  rstd = 1 / sqrt(mean(z^2) + eps);  y = z rstd (w + offset)
//   e4m3: s = max(largest |y| / 448, 2^-126) of a row or group, q = y / s
//
// A row is held in registers by a team of one to sixteen wavefronts, so it is
// read once: the sum of squares, the output and (for e4m3) the largest size
// all come from the registers, and a call is one launch.  A lane has four
// consecutive columns in each chunk of a row, or eight where every type is 16
// bits wide (16-byte accesses either way, contiguous over the wavefront).
//
// Bound by HBM from a few MB on: T = 16384, d = 2048 with a residual moves
// 268 MB in bf16 in 42.3 us (6.3 TB/s; a large copy reaches 5.3), 16381 x 2040
// from a 32-bit stream to e4m3 with a scale for 128 columns 369 MB in 64.3 us.
// A single row takes 2.2 us, most of it the launch.
#include <type_traits>

#include "norm.hpp"

namespace fff {
namespace {

// What goes past the caches: nothing, residual_out, or the inputs too.
enum { kStreamNone, kStreamResidual, kStreamAll };

template <typename X, typename S, bool F8, bool RAGGED, int STREAM, int WAVES, int C>
__global__ __launch_bounds__(block_threads(WAVES)) void rms_norm_kernel(NormArgs a) {
  constexpr int V = kCols<X, S>;
  constexpr int kTeam = WAVES * kWave;
  constexpr int kRows = block_threads(WAVES) / kTeam;  // rows a workgroup has at a time
  using At = Span<V, RAGGED>;
  __shared__ float lds_f[WAVES];
  __shared__ uint32_t lds_u[WAVES];
  const int lane = threadIdx.x % kTeam;
  const X* x = static_cast<const X*>(a.x);
  const S* r = static_cast<const S*>(a.residual);
  const X* w = static_cast<const X*>(a.weight);
  S* zout = static_cast<S*>(a.residual_out);
  const float offset = a.weight_offset + (w ? 0.0f : 1.0f);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (int64_t t = int64_t(blockIdx.x) * kRows + threadIdx.x / kTeam; t < a.T;
       t += int64_t(gridDim.x) * kRows) {
    const size_t row = static_cast<size_t>(t) * a.d;
    // What there is no tensor for is zeros (no weight: 1 with the offset).
    Pack<X, V> xr[C] = {}, wr[C] = {};
    Pack<S, V> rr[C] = {};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const At at((c * kTeam + lane) * V, a.d);
      if (x) at.template load<STREAM == kStreamAll>(xr[c], x + row);
      if (r) at.template load<STREAM == kStreamAll>(rr[c], r + row);
    }
    auto load_weight = [&]() {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (w) At((c * kTeam + lane) * V, a.d).template load<false>(wr[c], w);
    };
    // With the row if the registers hold it; eight chunks of one leave no room.
    if constexpr (C < 8) load_weight();
    float z[C][V];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const At at((c * kTeam + lane) * V, a.d);
#pragma unroll
      for (int i = 0; i < V; ++i) z[c][i] = xr[c].get(i) + rr[c].get(i);
      at.clear(z[c]);
#pragma unroll
      for (int i = 0; i < V; ++i) ss += z[c][i] * z[c][i];
      // y is formed from the 32-bit sum; only the stored copy is rounded.
      if (zout) at.template store<STREAM != kStreamNone>(packed<S, V>(z[c]), zout + row);
    }
    ss = team_total<WAVES>(ss, lds_f);
    if constexpr (C == 8) load_weight();
    const float rstd = 1.0f / sqrtf(ss * inv_d + a.eps);
    if (a.rstd && lane == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i)
        z[c][i] = z[c][i] * rstd * (wr[c].get(i) + offset);
    if constexpr (!F8) {
      X* y = static_cast<X*>(a.y);
#pragma unroll
      for (int c = 0; c < C; ++c)
        At((c * kTeam + lane) * V, a.d).store(packed<X, V>(z[c]), y + row);
    } else {
      uint8_t* y = static_cast<uint8_t*>(a.y);
      uint32_t top[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        top[c] = 0;
        // (once more: 0 times a NaN weight that the lane does not have)
        At((c * kTeam + lane) * V, a.d).clear(z[c]);
#pragma unroll
        for (int i = 0; i < V; ++i) top[c] = umax(top[c], size_bits(z[c][i]));
        // (a lane past the row's end: an infinite rstd has made its zeros NaN)
        if ((c * kTeam + lane) * V >= a.d) top[c] = 0;
      }
      if (a.group == 0) {
#pragma unroll
        for (int c = 1; c < C; ++c) top[0] = umax(top[0], top[c]);
        top[0] = team_max<WAVES>(top[0], lds_u);
#pragma unroll
        for (int c = 1; c < C; ++c) top[c] = top[0];
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * kTeam + lane) * V;
        if (a.group != 0) top[c] = group_top<V>(top[c], a.group);
        const float scale = e4m3_scale(top[c]);
        const float inv = reciprocal(scale);
#pragma unroll
        for (int i = 0; i < V; ++i) z[c][i] *= inv;
        if (col < a.d) {
          At(col, a.d).store(pack_e4m3(z[c]), y + row);
          if (a.group == 0) {
            if (col == 0) a.scale[t] = scale;
          } else if (col % a.group == 0) {
            a.scale[t * ((a.d + a.group - 1) / a.group) + col / a.group] = scale;
          }
        }
      }
    }
  }
}

// Forward: two chunks per lane as long as a row fits eight wavefronts.  At
// T = 16384, d = 2048 in bf16 2 x 2 takes 46.9 us, 4 x 1 49.1 and 1 x 4 48.2;
// at 4096 x 8192 8 x 2 takes 47.2 and 4 x 4 49.0.
template <int V, typename F>
void with_forward_plan(int pieces, const F& f) {
  if (pieces <= 1) f(Plan<1, 1>());
  else if (pieces <= 2) f(Plan<1, 2>());
  else if (pieces <= 4) f(Plan<2, 2>());
  else if (pieces <= 8) f(Plan<4, 2>());
  else if (pieces <= 16) f(Plan<8, 2>());
  else if (pieces <= 24) f(Plan<8, 3>());
  else if (pieces <= 32) f(Plan<8, 4>());
  else if (V == 8 || pieces <= 64) f(Plan<16, 4>());
  else if constexpr (V == 4) f(Plan<16, 8>());
}

// Of what a call reads and writes only y is used at once.  From 64 MB on
// residual_out, which the next norm reads, is written past the caches, and
// from 224 MB on the inputs are read past them too: both would push y out of
// the 256 MB last-level cache.  Together with a producer of x and a reader of
// y (us, nothing / residual_out / all past the caches):
//   bf16 16384 x 2048 (268 MB)   89.2 / 87.2 / 82.1   (the norm alone 46.7 / 46.8 / 42.3)
//   bf16 8192 x 2048 (134 MB)    45.2 / 44.2 / 44.1
//   bf16 4096 x 2048 (67 MB)     23.8 / 23.4 / 25.3
//   32 bits to e4m3, 8192 x 2040 (184 MB)   56.2 / 53.6 / 54.6
//   32 bits to e4m3, 4096 x 2040 (92 MB)    31.7 / 29.1 / 31.6
constexpr int64_t kStreamResidualBytes = int64_t(64) << 20;
constexpr int64_t kStreamInputBytes = int64_t(224) << 20;

template <typename X, typename S, bool F8>
hipError_t run_fwd(const NormArgs& a, hipStream_t st) {
  const int64_t bytes = a.T * a.d * ((a.x ? sizeof(X) : 0) + (a.residual ? sizeof(S) : 0) +
                                     (a.residual_out ? sizeof(S) : 0) + (F8 ? 1 : sizeof(X)));
  with_forward_plan<kCols<X, S>>(pieces_of(a.d, kCols<X, S>), [&](auto plan) {
    using P = decltype(plan);
    const RowPlan p = {P::kWaves, P::kChunks};
    const int64_t blocks = (a.T + p.rows() - 1) / p.rows();
    const int grid = static_cast<int>(blocks < (1 << 20) ? blocks : (1 << 20));
    auto launch = [&](auto ragged, auto stream) {
      rms_norm_kernel<X, S, F8, decltype(ragged)::value, decltype(stream)::value, P::kWaves,
                      P::kChunks><<<grid, p.threads(), 0, st>>>(a);
    };
    auto launch_ragged = [&](auto stream) {
      if (a.d % kCols<X, S> != 0)
        launch(std::true_type(), stream);
      else
        launch(std::false_type(), stream);
    };
    if (bytes >= kStreamInputBytes)
      launch_ragged(std::integral_constant<int, kStreamAll>());
    else if (bytes >= kStreamResidualBytes)
      launch_ragged(std::integral_constant<int, kStreamResidual>());
    else
      launch_ragged(std::integral_constant<int, kStreamNone>());
  });
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t st) {
  if (a.bf16 && a.stream_bf16)
    return a.e4m3 ? run_fwd<uint16_t, uint16_t, true>(a, st)
                  : run_fwd<uint16_t, uint16_t, false>(a, st);
  if (a.bf16)
    return a.e4m3 ? run_fwd<uint16_t, float, true>(a, st) : run_fwd<uint16_t, float, false>(a, st);
  return a.e4m3 ? run_fwd<float, float, true>(a, st) : run_fwd<float, float, false>(a, st);
}

}  // namespace fff
