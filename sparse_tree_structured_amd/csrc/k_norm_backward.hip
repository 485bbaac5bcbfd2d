// Backward pass of the root-mean-square norm:
//
//   g = dy (w + offset);  dz = rstd (g - z rstd mean(g z rstd)) + dres
//   dw = sum over rows of dy z rstd
//
// Rows are held as in the forward pass; a team takes every so many-th row and
// keeps its columns' share of dw in registers, so that dw costs one partial
// sum of d columns per workgroup and a second kernel that adds them in a fixed
// order (no atomics: the same bits on every call).
//
// Bound by HBM: T = 16384, d = 2048 in bf16 with the residual's gradient moves
// 268 MB in 44 us and adds 512 partials in 4 us.  With few rows the two
// launches are what counts.
#include <type_traits>

#include "norm.hpp"

namespace fff {
namespace {

// R rows at a time per team, whose dots share a barrier; the columns' share
// of dw stays in registers over the team's rows and goes to the workspace
// once per workgroup.
template <typename X, typename S, bool RAGGED, int WAVES, int C, int R, bool STREAM>
__global__ __launch_bounds__(block_threads(WAVES)) void rms_norm_backward_kernel(NormGradArgs a) {
  constexpr int V = kCols<X, S>;
  constexpr int kTeam = WAVES * kWave;
  constexpr int kRows = block_threads(WAVES) / kTeam;
  using At = Span<V, RAGGED>;
  // Beside a dx of another type, which the next operator reads, dz waits for
  // the norm before.
  constexpr bool kStreamDz = STREAM && !std::is_same<X, S>::value;
  // Two sets, used in turn: a wavefront that is a round ahead writes the
  // other one, and the round's barrier keeps it from being two ahead.
  __shared__ float lds[2][R][WAVES];
  const int lane = threadIdx.x % kTeam;
  const X* dy = static_cast<const X*>(a.dy);
  const S* zin = static_cast<const S*>(a.z);
  const X* w = static_cast<const X*>(a.weight);
  const S* dres = static_cast<const S*>(a.dresidual);
  S* dz = static_cast<S*>(a.dz);
  X* dx = static_cast<X*>(a.dx);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float gain[C][V], acc[C][V];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const At at((c * kTeam + lane) * V, a.d);
    Pack<X, V> wr = {};
    if (w) at.template load<false>(wr, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      gain[c][i] = wr.get(i) + a.weight_offset + (w ? 0.0f : 1.0f);
      acc[c][i] = 0.0f;
    }
    at.clear(gain[c]);  // zero times an infinite weight would be NaN in the dot
  }
  const int64_t stride = int64_t(gridDim.x) * kRows;
  int set = 0;
  for (int64_t t0 = int64_t(blockIdx.x) * kRows + threadIdx.x / kTeam; t0 < a.T;
       t0 += R * stride, set ^= 1) {
    Pack<X, V> yr[R][C];
    Pack<S, V> zr[R][C], er[R][C] = {};
    float rstd[R], dot[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t t = t0 + k * stride;
      const size_t row = static_cast<size_t>(t) * a.d;
      rstd[k] = t < a.T ? a.rstd[t] : 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const At at((c * kTeam + lane) * V, a.d);
        yr[k][c] = Pack<X, V>();
        zr[k][c] = Pack<S, V>();
        if (t >= a.T) continue;  // a row past the last one is zeros
        at.template load<STREAM>(yr[k][c], dy + row);
        at.template load<STREAM>(zr[k][c], zin + row);
        if (dres) at.template load<STREAM>(er[k][c], dres + row);
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      dot[k] = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = yr[k][c].get(i);
        At((c * kTeam + lane) * V, a.d).clear(d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float zh = zr[k][c].get(i) * rstd[k];
          acc[c][i] += d[i] * zh;
          dot[k] += d[i] * gain[c][i] * zh;
        }
      }
      dot[k] = wave_total(dot[k]);
    }
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
        for (int k = 0; k < R; ++k) lds[set][k][threadIdx.x / kWave] = dot[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < R; ++k) {
        dot[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) dot[k] += lds[set][k][i];
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t t = t0 + k * stride;
      const size_t row = static_cast<size_t>(t) * a.d;
      const float mean = dot[k] * inv_d;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const At at((c * kTeam + lane) * V, a.d);
        if (t >= a.T) continue;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float zh = zr[k][c].get(i) * rstd[k];
          v[i] = rstd[k] * (yr[k][c].get(i) * gain[c][i] - zh * mean) + er[k][c].get(i);
        }
        at.template store<kStreamDz>(packed<S, V>(v), dz + row);
        if (dx) at.store(packed<X, V>(v), dx + row);
      }
    }
  }
  if (!a.partial) return;
  if constexpr (kRows > 1) {  // the workgroup's teams as one partial sum
    __shared__ float sums[kRows][C * V][kTeam];
    const int team = threadIdx.x / kTeam;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) sums[team][c * V + i][lane] = acc[c][i];
    __syncthreads();
    if (team != 0) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 1; k < kRows; ++k) acc[c][i] += sums[k][c * V + i][lane];
  }
  float* out = a.partial + size_t(blockIdx.x) * a.d;
#pragma unroll
  for (int c = 0; c < C; ++c) At((c * kTeam + lane) * V, a.d).store_floats(acc[c], out);
}

// dw[j] = sum over the partials in a fixed order: 32 columns (a 128-byte line
// of every partial) per workgroup, 32 slices of the partials, sixteen loads
// in flight per lane, the slices joined in LDS.
constexpr int kSumCols = 32, kSumSlices = 32;

__global__ __launch_bounds__(kSumCols * kSumSlices) void rms_norm_dweight_kernel(
    const float* partial, int count, int d, float* dw) {
  __shared__ float lds[kSumSlices][kSumCols + 1];
  const int lane = threadIdx.x % kSumCols;
  const int col = blockIdx.x * kSumCols + lane;
  const int slice = threadIdx.x / kSumCols;
  float s = 0.0f;
  if (col < d) {
    const float* p = partial + col;
    for (int i = slice; i < count; i += 16 * kSumSlices) {
      float v[16];
#pragma unroll
      for (int k = 0; k < 16; ++k)
        v[k] = i + k * kSumSlices < count ? p[size_t(i + k * kSumSlices) * d] : 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) s += v[k];
    }
  }
  lds[slice][lane] = s;
  __syncthreads();
  if (threadIdx.x < kSumCols && col < d) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumSlices; ++i) s += lds[i][threadIdx.x];
    dw[col] = s;
  }
}

// Small batches, and the widest rows, in one launch without a workspace: the
// first a.rows workgroups have the rows of dz (all of them, or none), and the
// others 32 columns of dw each, for which they read dy and z once more (dw
// needs no row's dot).
constexpr int kSmallCols = 32;

template <typename X, typename S, bool RAGGED, int THREADS, int C>
__global__ __launch_bounds__(THREADS) void rms_norm_backward_rows_columns_kernel(NormGradArgs a) {
  constexpr int V = kCols<X, S>;
  const X* dy = static_cast<const X*>(a.dy);
  const S* zin = static_cast<const S*>(a.z);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  if (static_cast<int>(blockIdx.x) < a.rows) {
    using At = Span<V, RAGGED>;
    __shared__ float lds[THREADS / kWave];
    const X* w = static_cast<const X*>(a.weight);
    const S* dres = static_cast<const S*>(a.dresidual);
    S* dz = static_cast<S*>(a.dz);
    X* dx = static_cast<X*>(a.dx);
    const float offset = a.weight_offset + (w ? 0.0f : 1.0f);
    for (int64_t t = blockIdx.x; t < a.T; t += a.rows) {
      const size_t row = static_cast<size_t>(t) * a.d;
      const float rstd = a.rstd[t];
      Pack<X, V> yr[C], wr[C] = {};
      Pack<S, V> zr[C], er[C] = {};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const At at((c * THREADS + threadIdx.x) * V, a.d);
        at.template load<false>(yr[c], dy + row);
        at.template load<false>(zr[c], zin + row);
        if (w) at.template load<false>(wr[c], w);
        if (dres) at.template load<false>(er[c], dres + row);
      }
      float g[C][V], dot = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < V; ++i) g[c][i] = yr[c].get(i) * (wr[c].get(i) + offset);
        At((c * THREADS + threadIdx.x) * V, a.d).clear(g[c]);
#pragma unroll
        for (int i = 0; i < V; ++i) dot += g[c][i] * (zr[c].get(i) * rstd);
      }
      dot = team_total<THREADS / kWave>(dot, lds) * inv_d;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const At at((c * THREADS + threadIdx.x) * V, a.d);
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
          v[i] = rstd * (g[c][i] - zr[c].get(i) * rstd * dot) + er[c].get(i);
        at.store(packed<S, V>(v), dz + row);
        if (dx) at.store(packed<X, V>(v), dx + row);
      }
    }
    return;
  }
  // Slices of the rows by eight lanes of four columns.
  constexpr int kLanes = kSmallCols / 4, kSlices = THREADS / kLanes;
  __shared__ float sums[kSlices][kSmallCols + 1];
  const int lane = threadIdx.x % kLanes, slice = threadIdx.x / kLanes;
  const int first = (static_cast<int>(blockIdx.x) - a.rows) * kSmallCols;
  const int col = first + lane * 4;
  float s[4] = {};
#pragma unroll 4
  for (int64_t t = slice; t < a.T; t += kSlices) {
    Pack<X, 4> y;
    Pack<S, 4> z;
    y.load(dy + t * a.d + col, a.d - col);
    z.load(zin + t * a.d + col, a.d - col);
    const float rstd = a.rstd[t];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += y.get(i) * (z.get(i) * rstd);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sums[slice][lane * 4 + i] = s[i];
  __syncthreads();
  const int mine = first + threadIdx.x;
  if (threadIdx.x < kSmallCols && mine < a.d) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) v += sums[i][threadIdx.x];
    a.dweight[mine] = v;
  }
}

// Backward: one chunk per lane up to four wavefronts, whose dots then share
// a barrier for two rows.
template <int V, typename F>
void with_backward_plan(int pieces, const F& f) {
  if (pieces <= 1) f(Plan<1, 1>());
  else if (pieces <= 2) f(Plan<2, 1>());
  else if (pieces <= 3) f(Plan<3, 1>());
  else if (pieces <= 4) f(Plan<4, 1>());
  else if (pieces <= 6) f(Plan<3, 2>());
  else if (pieces <= 8) f(Plan<4, 2>());
  else if (pieces <= 12) f(Plan<4, 3>());
  else if (pieces <= 16) f(Plan<4, 4>());
  else if (pieces <= 24) f(Plan<8, 3>());
  else if (V == 8 || pieces <= 32) f(Plan<8, 4>());
  else if constexpr (V == 4) f(Plan<16, 4>());
}

// Rows of the backward at a time: two where a lane has one chunk of each.
constexpr int grad_rows(int chunks) { return chunks == 1 ? 2 : 1; }

// Workgroups of the backward: as many as keep about 48 KB of loads in flight
// on each of the 256 compute units (every one more is another partial sum of
// d columns to write and read), but two per compute unit, or one of more than
// four wavefronts.  At T = 16384, d = 2048 (bf16) 512 workgroups take 48.6 us
// with the sum of the partials, 256 take 61.4 and 1024 54.1; at 8000 x 5000
// 512 take 71.5, 256 90.2 and 1024 76.3; at 3000 x 12288 256 take 65.5, 512
// 72.2.
int grad_grid(int64_t T, const RowPlan& p) {
  constexpr int kComputeUnits = 256;
  const int64_t blocks = (T + p.rows() - 1) / p.rows();
  const int least = p.waves > 4 ? kComputeUnits : 2 * kComputeUnits;
  int most = 16 * kComputeUnits / (p.threads() / kWave * p.chunks * grad_rows(p.chunks));
  if (most < least) most = least;
  return static_cast<int>(blocks < most ? blocks : most);
}

// From this many bytes of inputs on they are read past the caches: they would
// push out one another and the dz that the next operator reads.  At
// T = 16384, d = 2048 in bf16 (201 MB) that takes 54.3 us instead of 56.5,
// and with a reader of dz behind it 71.0 instead of 77.5; at T = 4096, where
// the inputs fit the 256 MB last-level cache, it takes 22.2 instead of 19.5.
// A 32-bit dz beside a bf16 dx is then written past them too: with a producer
// of dy and a reader of dx 122.0 us instead of 136.2.
constexpr int64_t kGradStreamBytes = int64_t(160) << 20;

// Whether a batch goes through the one-launch kernel.  Up to 1024 rows and
// 16 MB of dy and z it does: 512 x 2048 takes 12.1 us a call instead of 17.1,
// 512 x 8192 12.1 instead of 17.2; the few slices of a dw column make it slow
// for many rows (2048 x 2048 would take 21.7 us instead of 17.0, 8000 x 100 64
// instead of 19).  So do rows of more than 16384 columns, for which the other
// kernel would have more than 16 columns of dw to a lane and one workgroup to
// a compute unit: 3000 x 20000 in bf16 158 us instead of 345, 1000 x 32768 in
// 32 bits 180 instead of 228 (at 12288 columns 171 instead of 103).
constexpr int64_t kSmallRows = 1024, kSmallBytes = int64_t(16) << 20;
constexpr int kWide = 16384;

template <typename X, typename S>
bool one_launch(int64_t T, int d) {
  return d > kWide ||
         (T <= kSmallRows && T * d * int64_t(sizeof(X) + sizeof(S)) <= kSmallBytes);
}

bool overlap(const void* p, int64_t np, const void* q, int64_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + nq && b < a + np;
}

template <typename X, typename S, int THREADS, int C>
void launch_rows_and_columns(const NormGradArgs& args, hipStream_t st) {
  NormGradArgs a = args;
  const int columns = a.dweight ? (a.d + kSmallCols - 1) / kSmallCols : 0;
  auto launch = [&](int rows, int columns) {  // workgroups
    a.rows = rows;
    if (a.d % kCols<X, S> != 0)
      rms_norm_backward_rows_columns_kernel<X, S, true, THREADS, C>
          <<<rows + columns, THREADS, 0, st>>>(a);
    else
      rms_norm_backward_rows_columns_kernel<X, S, false, THREADS, C>
          <<<rows + columns, THREADS, 0, st>>>(a);
  };
  // Where dz or dx takes the place of dy or z, dw has to read them first.
  const int64_t nx = a.T * a.d * sizeof(X), ns = a.T * a.d * sizeof(S);
  const int rows = static_cast<int>(a.T < (1 << 20) ? a.T : (1 << 20));
  if (columns > 0 && (overlap(a.dz, ns, a.dy, nx) || overlap(a.dz, ns, a.z, ns) ||
                      overlap(a.dx, nx, a.dy, nx) || overlap(a.dx, nx, a.z, ns))) {
    launch(0, columns);
    launch(rows, 0);
  } else {
    launch(rows, columns);
  }
}

template <typename X, typename S>
size_t partials(int64_t T, int d) {
  if (one_launch<X, S>(T, d)) return 0;
  size_t rows = 0;
  with_backward_plan<kCols<X, S>>(pieces_of(d, kCols<X, S>), [&](auto plan) {
    const RowPlan p = {decltype(plan)::kWaves, decltype(plan)::kChunks};
    rows = T == 0 ? 0 : grad_grid(T, p);
  });
  return rows;
}

template <typename X, typename S>
hipError_t run_bwd(const NormGradArgs& a, hipStream_t st) {
  if (one_launch<X, S>(a.T, a.d)) {
    const int pieces = pieces_of(a.d, kCols<X, S>);
    if (pieces <= 4)
      launch_rows_and_columns<X, S, 256, 1>(a, st);
    else if (pieces <= 8)
      launch_rows_and_columns<X, S, 256, 2>(a, st);
    else if (pieces <= 16)
      launch_rows_and_columns<X, S, 256, 4>(a, st);
    else if (pieces <= 32)
      launch_rows_and_columns<X, S, 512, 4>(a, st);
    else if (pieces <= 64)
      launch_rows_and_columns<X, S, 1024, 4>(a, st);
    else if constexpr (kCols<X, S> == 4)
      launch_rows_and_columns<X, S, 1024, 8>(a, st);
    return hipGetLastError();
  }
  with_backward_plan<kCols<X, S>>(pieces_of(a.d, kCols<X, S>), [&](auto plan) {
    using P = decltype(plan);
    constexpr int R = grad_rows(P::kChunks);
    const RowPlan p = {P::kWaves, P::kChunks};
    const int64_t bytes = a.T * a.d * (sizeof(X) + sizeof(S) * (a.dresidual ? 2 : 1));
    auto launch = [&](auto ragged, auto stream) {
      rms_norm_backward_kernel<X, S, decltype(ragged)::value, P::kWaves, P::kChunks, R,
                               decltype(stream)::value>
          <<<grad_grid(a.T, p), p.threads(), 0, st>>>(a);
    };
    const bool ragged = a.d % kCols<X, S> != 0, stream = bytes >= kGradStreamBytes;
    if (ragged && stream) launch(std::true_type(), std::true_type());
    else if (ragged) launch(std::true_type(), std::false_type());
    else if (stream) launch(std::false_type(), std::true_type());
    else launch(std::false_type(), std::false_type());
  });
  return hipGetLastError();
}

}  // namespace

size_t rms_norm_backward_partials(int64_t T, int d, bool bf16, bool stream_bf16) {
  return bf16 && stream_bf16 ? partials<uint16_t, uint16_t>(T, d)
         : bf16              ? partials<uint16_t, float>(T, d)
                             : partials<float, float>(T, d);
}

hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t st) {
  if (a.T > 0) {
    const hipError_t e = a.bf16 && a.stream_bf16 ? run_bwd<uint16_t, uint16_t>(a, st)
                         : a.bf16                ? run_bwd<uint16_t, float>(a, st)
                                                 : run_bwd<float, float>(a, st);
    if (e != hipSuccess) return e;
  }
  const int count = static_cast<int>(rms_norm_backward_partials(a.T, a.d, a.bf16, a.stream_bf16));
  if (!a.dweight || (a.T > 0 && count == 0)) return hipSuccess;  // one launch has written dw
  rms_norm_dweight_kernel<<<(a.d + kSumCols - 1) / kSumCols, kSumCols * kSumSlices, 0, st>>>(
      a.partial, count, a.d, a.dweight);
  return hipGetLastError();
}

}  // namespace fff
