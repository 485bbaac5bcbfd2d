// Root-mean-square norm of rows with the residual's addition, its output in
// the layer's type or in e4m3 with scales, and its backward pass.
//
//   z = x + r;  rstd = 1 / sqrt(mean(z^2) + eps);  y = z rstd (w + offset)
//   g = dy (w + offset);  dz = rstd (g - z rstd mean(g z rstd)) + dres
//   dw = sum over rows of dy z rstd
//
// A row is held in registers by a team of one to sixteen wavefronts, so it is
// read once: the sum of squares, the output and (for e4m3) the largest size
// all come from the registers.  A lane has four consecutive columns in each
// chunk of a row, or eight where every type is 16 bits wide (16-byte accesses
// either way, contiguous over the wavefront).
#include "common.hpp"
#include "launch_train.hpp"
#include "train.hpp"

namespace fff {
namespace {

// Sum of v over a team of WAVES wavefronts (one per workgroup when WAVES > 1).
template <int WAVES>
__device__ __forceinline__ float team_total(float v, float* lds) {
  v = wave_total(v);
  if constexpr (WAVES > 1) {
    const int wave = threadIdx.x / kWave;
    __syncthreads();  // the previous row's totals have been read
    if ((threadIdx.x & (kWave - 1)) == 0) lds[wave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) v += lds[i];
  }
  return v;
}

template <int WAVES>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* lds) {
  v = wave_max(v);
  if constexpr (WAVES > 1) {
    const int wave = threadIdx.x / kWave;
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0) lds[wave] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) v = umax(v, lds[i]);
  }
  return v;
}

constexpr int block_threads(int waves) { return waves == 1 ? 4 * kWave : waves * kWave; }

// Columns of a lane in one chunk.
template <typename X, typename S>
constexpr int kCols = sizeof(X) == 2 && sizeof(S) == 2 ? 8 : 4;

// The columns of one chunk of a row that a lane has.  Where d is a multiple
// of V (not RAGGED) that is all V or none.
template <int V, bool RAGGED>
struct Span {
  int first;
  bool in;
  __device__ __forceinline__ Span(int first, int d) : first(first), in(first < d) {}
  template <bool STREAM, typename E>
  __device__ __forceinline__ void load(Pack<E, V>& p, const E* row) const {
    p = Pack<E, V>();
    if (in) p.template load<STREAM>(row + first, V);
  }
  __device__ __forceinline__ void clear(float (&)[V]) const {}
  template <typename E>
  __device__ __forceinline__ void store(const Pack<E, V>& p, E* row) const {
    if (in) p.store(row + first, V);
  }
  __device__ __forceinline__ void store_floats(const float (&v)[V], float* row) const {
    if (!in) return;
#pragma unroll
    for (int h = 0; h < V; h += 4) {
      const float four[4] = {v[h], v[h + 1], v[h + 2], v[h + 3]};
      packed<float, 4>(four).store(row + first + h, 4);
    }
  }
};

// Otherwise columns col + lo .. col + hi - 1 (nothing where lo = V).  An
// access that would leave the row is moved back to end with it, so that every
// load is a whole one inside the row and none waits for a short one (at
// 8000 x 2703 in bf16 the forward takes 40.7 us instead of 53.6); what the
// lane then has twice, below lo, counts for nothing and is not stored.
template <int V>
struct Span<V, true> {
  int col, lo, hi;
  __device__ __forceinline__ Span(int first, int d) {
    const int last = d >= V ? d - V : 0;
    col = first < last ? first : last;
    lo = first - col < V ? first - col : V;
    hi = d >= V ? V : d;
    if (d < V && first > 0) lo = V;
  }
  __device__ __forceinline__ bool has(int i) const { return i >= lo && i < hi; }
  template <bool STREAM, typename E>
  __device__ __forceinline__ void load(Pack<E, V>& p, const E* row) const {
    p.template load<STREAM>(row + col, hi);
  }
  // Zeros in place of what the lane does not have.
  __device__ __forceinline__ void clear(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = has(i) ? v[i] : 0.0f;
  }
  template <typename E>
  __device__ __forceinline__ void store(const Pack<E, V>& p, E* row) const {
    if (lo == 0 && hi == V)
      p.store(row + col, V);
    else
      p.store_range(row + col, lo, hi);
  }
  __device__ __forceinline__ void store_floats(const float (&v)[V], float* row) const {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (has(i)) row[col + i] = v[i];
  }
};

// Lanes of one scale's group.
template <int V>
__device__ __forceinline__ uint32_t group_top(uint32_t v, int group) {
  if (group == 32) return group_max<32 / V>(v);
  if (group == 64) return group_max<64 / V>(v);
  return group_max<128 / V>(v);
}

template <typename X, typename S, bool F8, bool RAGGED, int WAVES, int C>
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
      if (x) at.template load<false>(xr[c], x + row);
      if (r) at.template load<false>(rr[c], r + row);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const At at((c * kTeam + lane) * V, a.d);
      if (w) at.template load<false>(wr[c], w);
    }
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
      if (zout) at.store(packed<S, V>(z[c]), zout + row);
    }
    ss = team_total<WAVES>(ss, lds_f);
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

// R rows at a time per team, whose dots share a barrier; the columns' share
// of dw stays in registers over the team's rows and goes to the workspace
// once per team.
template <typename X, typename S, bool RAGGED, int WAVES, int C, int R, bool STREAM>
__global__ __launch_bounds__(block_threads(WAVES)) void rms_norm_backward_kernel(NormGradArgs a) {
  constexpr int V = kCols<X, S>;
  constexpr int kTeam = WAVES * kWave;
  constexpr int kRows = block_threads(WAVES) / kTeam;
  using At = Span<V, RAGGED>;
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
        at.store(packed<S, V>(v), dz + row);
        if (dx) at.store(packed<X, V>(v), dx + row);
      }
    }
  }
  if (!a.partial) return;
  float* out = a.partial + (size_t(blockIdx.x) * kRows + threadIdx.x / kTeam) * a.d;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    At((c * kTeam + lane) * V, a.d).store_floats(acc[c], out);
  }
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

// Wavefronts of a row and chunks of each.
struct RowPlan {
  int waves, chunks;
  int rows() const { return waves == 1 ? 4 : 1; }  // of a workgroup
  int threads() const { return block_threads(waves); }
};

// Accesses of one wavefront that a row takes.
int pieces_of(int d, int cols) { return (d + cols * kWave - 1) / (cols * kWave); }

template <int W, int C> struct Plan {
  static constexpr int kWaves = W, kChunks = C;
};

// Forward: two chunks per lane as long as a row fits eight wavefronts.  At
// T = 16384, d = 2048 in bf16 2 x 2 takes 46.9 us, 4 x 1 49.1 and 1 x 4 48.2;
// at 4096 x 8192 8 x 2 takes 47.2 and 4 x 4 49.0.
template <typename F>
void with_forward_plan(int pieces, const F& f) {
  if (pieces <= 1) f(Plan<1, 1>());
  else if (pieces <= 2) f(Plan<1, 2>());
  else if (pieces <= 4) f(Plan<2, 2>());
  else if (pieces <= 8) f(Plan<4, 2>());
  else if (pieces <= 16) f(Plan<8, 2>());
  else if (pieces <= 32) f(Plan<8, 4>());
  else if (pieces <= 64) f(Plan<16, 4>());
  else f(Plan<16, 8>());
}

template <typename X, typename S, bool F8>
hipError_t run_fwd(const NormArgs& a, hipStream_t st) {
  with_forward_plan(pieces_of(a.d, kCols<X, S>), [&](auto plan) {
    using P = decltype(plan);
    const RowPlan p = {P::kWaves, P::kChunks};
    const int64_t blocks = (a.T + p.rows() - 1) / p.rows();
    const int grid = static_cast<int>(blocks < (1 << 20) ? blocks : (1 << 20));
    if (a.d % kCols<X, S> != 0)
      rms_norm_kernel<X, S, F8, true, P::kWaves, P::kChunks><<<grid, p.threads(), 0, st>>>(a);
    else
      rms_norm_kernel<X, S, F8, false, P::kWaves, P::kChunks><<<grid, p.threads(), 0, st>>>(a);
  });
  return hipGetLastError();
}

// Backward: one chunk per lane up to four wavefronts, whose dots then share
// a barrier for two rows.
template <typename F>
void with_backward_plan(int pieces, const F& f) {
  if (pieces <= 1) f(Plan<1, 1>());
  else if (pieces <= 2) f(Plan<2, 1>());
  else if (pieces <= 3) f(Plan<3, 1>());
  else if (pieces <= 4) f(Plan<4, 1>());
  else if (pieces <= 6) f(Plan<3, 2>());
  else if (pieces <= 8) f(Plan<4, 2>());
  else if (pieces <= 16) f(Plan<4, 4>());
  else if (pieces <= 32) f(Plan<8, 4>());
  else if (pieces <= 64) f(Plan<16, 4>());
  else f(Plan<16, 8>());
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
constexpr int64_t kGradStreamBytes = int64_t(160) << 20;

int cols_of(bool bf16, bool stream_bf16) {
  return bf16 && stream_bf16 ? kCols<uint16_t, uint16_t> : kCols<float, float>;
}

template <typename X, typename S>
hipError_t run_bwd(const NormGradArgs& a, hipStream_t st) {
  with_backward_plan(pieces_of(a.d, kCols<X, S>), [&](auto plan) {
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

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t st) {
  if (a.bf16 && a.stream_bf16)
    return a.e4m3 ? run_fwd<uint16_t, uint16_t, true>(a, st)
                  : run_fwd<uint16_t, uint16_t, false>(a, st);
  if (a.bf16)
    return a.e4m3 ? run_fwd<uint16_t, float, true>(a, st) : run_fwd<uint16_t, float, false>(a, st);
  return a.e4m3 ? run_fwd<float, float, true>(a, st) : run_fwd<float, float, false>(a, st);
}

size_t rms_norm_backward_partials(int64_t T, int d, bool bf16, bool stream_bf16) {
  size_t rows = 0;
  with_backward_plan(pieces_of(d, cols_of(bf16, stream_bf16)), [&](auto plan) {
    const RowPlan p = {decltype(plan)::kWaves, decltype(plan)::kChunks};
    rows = T == 0 ? 0 : size_t(grad_grid(T, p)) * p.rows();
  });
  return rows;
}

hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t st) {
  if (a.T > 0) {
    const hipError_t e = a.bf16 && a.stream_bf16 ? run_bwd<uint16_t, uint16_t>(a, st)
                         : a.bf16                ? run_bwd<uint16_t, float>(a, st)
                                                 : run_bwd<float, float>(a, st);
    if (e != hipSuccess) return e;
  }
  if (!a.dweight) return hipSuccess;
  const int count = static_cast<int>(rms_norm_backward_partials(a.T, a.d, a.bf16, a.stream_bf16));
  rms_norm_dweight_kernel<<<(a.d + kSumCols - 1) / kSumCols, kSumCols * kSumSlices, 0, st>>>(
      a.partial, count, a.d, a.dweight);
  return hipGetLastError();
}

}  // namespace fff
