// Root-mean-square norm of rows with the residual's addition, its output in
// the layer's type or in e4m3 with scales, and its backward pass.
//
//   z = x + r;  rstd = 1 / sqrt(mean(z^2) + eps);  y = z rstd (w + offset)
//   g = dy (w + offset);  dz = rstd (g - z rstd mean(g z rstd)) + dres
//   dw = sum over rows of dy z rstd
//
// A row is held in registers by a team of one to sixteen wavefronts, eight
// consecutive columns per lane and chunk, so it is read once: the sum of
// squares, the output and (for e4m3) the largest size all come from the
// registers.
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

template <typename X, typename S, bool F8, int WAVES, int C>
__global__ __launch_bounds__(block_threads(WAVES)) void rms_norm_kernel(NormArgs a) {
  constexpr int kTeam = WAVES * kWave;
  constexpr int kRows = block_threads(WAVES) / kTeam;  // rows a workgroup has at a time
  __shared__ float lds_f[WAVES];
  __shared__ uint32_t lds_u[WAVES];
  const int lane = threadIdx.x % kTeam;
  const X* x = static_cast<const X*>(a.x);
  const S* r = static_cast<const S*>(a.residual);
  const X* w = static_cast<const X*>(a.weight);
  S* zout = static_cast<S*>(a.residual_out);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (int64_t t = int64_t(blockIdx.x) * kRows + threadIdx.x / kTeam; t < a.T;
       t += int64_t(gridDim.x) * kRows) {
    const size_t row = static_cast<size_t>(t) * a.d;
    Eight<X> xr[C], wr[C];
    Eight<S> rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * kTeam + lane) * 8;
      if (x) load_eight(xr[c], x + row + col, a.d - col);
      if (r) load_eight(rr[c], r + row + col, a.d - col);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * kTeam + lane) * 8;
      if (w) load_eight(wr[c], w + col, a.d - col);
    }
    float z[C][8];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * kTeam + lane) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[c][i] = (x ? xr[c].get(i) : 0.0f) + (r ? rr[c].get(i) : 0.0f);
        ss += z[c][i] * z[c][i];
      }
      // y is formed from the 32-bit sum; only the stored copy is rounded.
      if (zout) store_eight(zout + row + col, a.d - col, z[c]);
    }
    ss = team_total<WAVES>(ss, lds_f);
    const float rstd = 1.0f / sqrtf(ss * inv_d + a.eps);
    if (a.rstd && lane == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        z[c][i] = z[c][i] * rstd * ((w ? wr[c].get(i) : 1.0f) + a.weight_offset);
    if constexpr (!F8) {
      X* y = static_cast<X*>(a.y);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * kTeam + lane) * 8;
        store_eight(y + row + col, a.d - col, z[c]);
      }
    } else {
      uint8_t* y = static_cast<uint8_t*>(a.y);
      uint32_t top[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * kTeam + lane) * 8;
        top[c] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < a.d) top[c] = umax(top[c], size_bits(z[c][i]));
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
        const int col = (c * kTeam + lane) * 8;
        if (a.group == 32) top[c] = group_max<4>(top[c]);
        if (a.group == 64) top[c] = group_max<8>(top[c]);
        if (a.group == 128) top[c] = group_max<16>(top[c]);
        const float scale = e4m3_scale(top[c]);
        const float inv = 1.0f / scale;
#pragma unroll
        for (int i = 0; i < 8; ++i) z[c][i] *= inv;
        if (col < a.d) {
          store_packed(y + row + col, a.d - col, pack_e4m3(z[c]));
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

// One row at a time per team; the columns' share of dw stays in registers
// over the team's rows and goes to the workspace once per workgroup.
template <typename X, typename S, int WAVES, int C>
__global__ __launch_bounds__(block_threads(WAVES)) void rms_norm_backward_kernel(NormGradArgs a) {
  constexpr int kTeam = WAVES * kWave;
  constexpr int kRows = block_threads(WAVES) / kTeam;
  __shared__ float lds_f[WAVES];
  const int lane = threadIdx.x % kTeam;
  const X* dy = static_cast<const X*>(a.dy);
  const S* zin = static_cast<const S*>(a.z);
  const X* w = static_cast<const X*>(a.weight);
  const S* dres = static_cast<const S*>(a.dresidual);
  S* dz = static_cast<S*>(a.dz);
  X* dx = static_cast<X*>(a.dx);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float gain[C][8], acc[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * kTeam + lane) * 8;
    Eight<X> wr;
    if (w) load_eight(wr, w + col, a.d - col);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gain[c][i] = (w ? wr.get(i) : 1.0f) + a.weight_offset;
      acc[c][i] = 0.0f;
    }
  }
  for (int64_t t = int64_t(blockIdx.x) * kRows + threadIdx.x / kTeam; t < a.T;
       t += int64_t(gridDim.x) * kRows) {
    const size_t row = static_cast<size_t>(t) * a.d;
    const float rstd = a.rstd[t];
    Eight<X> yr[C];
    Eight<S> zr[C], er[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * kTeam + lane) * 8;
      load_eight(yr[c], dy + row + col, a.d - col);
      load_eight(zr[c], zin + row + col, a.d - col);
      if (dres) load_eight(er[c], dres + row + col, a.d - col);
    }
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float zh = zr[c].get(i) * rstd;
        const float d = yr[c].get(i);
        acc[c][i] += d * zh;
        dot += d * gain[c][i] * zh;
      }
    dot = team_total<WAVES>(dot, lds_f) * inv_d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * kTeam + lane) * 8;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float zh = zr[c].get(i) * rstd;
        v[i] = rstd * (yr[c].get(i) * gain[c][i] - zh * dot) + (dres ? er[c].get(i) : 0.0f);
      }
      store_eight(dz + row + col, a.d - col, v);
      if (dx) store_eight(dx + row + col, a.d - col, v);
    }
  }
  if (!a.partial) return;
  // A workgroup of several teams stores a partial sum for each.
  float* out = a.partial + (size_t(blockIdx.x) * kRows + threadIdx.x / kTeam) * a.d;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * kTeam + lane) * 8;
    store_eight(out + col, a.d - col, acc[c]);
  }
}

// dw[j] = sum over the partials in a fixed order: 16 columns (one 64-byte
// piece of every partial) per workgroup, 64 slices of the partials, sixteen
// loads in flight per lane, the slices joined in LDS.
constexpr int kSumCols = 16, kSumSlices = 64;

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

template <typename X, typename S, bool F8, int WAVES, int C>
hipError_t launch_fwd(const NormArgs& a, hipStream_t st) {
  constexpr int kRows = block_threads(WAVES) / (WAVES * kWave);
  const int64_t blocks = (a.T + kRows - 1) / kRows;
  const int grid = static_cast<int>(blocks < (1 << 20) ? blocks : (1 << 20));
  rms_norm_kernel<X, S, F8, WAVES, C><<<grid, block_threads(WAVES), 0, st>>>(a);
  return hipGetLastError();
}

template <typename X, typename S, bool F8>
hipError_t pick_fwd(const NormArgs& a, hipStream_t st) {
  if (a.d <= 512) return launch_fwd<X, S, F8, 1, 1>(a, st);
  if (a.d <= 2048) return launch_fwd<X, S, F8, 4, 1>(a, st);
  if (a.d <= 4096) return launch_fwd<X, S, F8, 4, 2>(a, st);
  if (a.d <= 8192) return launch_fwd<X, S, F8, 4, 4>(a, st);
  return launch_fwd<X, S, F8, 16, 4>(a, st);
}

struct GradPlan {
  int waves, chunks, rows, grid;  // rows: teams per workgroup
};

GradPlan grad_plan(int64_t T, int d) {
  GradPlan p;
  p.waves = d <= 512 ? 1 : d <= 8192 ? 4 : 16;
  p.chunks = d <= 2048 ? 1 : d <= 4096 ? 2 : 4;
  p.rows = p.waves == 1 ? 4 : 1;
  const int64_t blocks = (T + p.rows - 1) / p.rows;
  p.grid = static_cast<int>(blocks < 1024 ? blocks : 1024);
  return p;
}

template <typename X, typename S>
hipError_t run_bwd(const NormGradArgs& a, const GradPlan& p, hipStream_t st) {
  const int threads = block_threads(p.waves);
  if (p.waves == 1)
    rms_norm_backward_kernel<X, S, 1, 1><<<p.grid, threads, 0, st>>>(a);
  else if (p.waves == 4 && p.chunks == 1)
    rms_norm_backward_kernel<X, S, 4, 1><<<p.grid, threads, 0, st>>>(a);
  else if (p.waves == 4 && p.chunks == 2)
    rms_norm_backward_kernel<X, S, 4, 2><<<p.grid, threads, 0, st>>>(a);
  else if (p.waves == 4)
    rms_norm_backward_kernel<X, S, 4, 4><<<p.grid, threads, 0, st>>>(a);
  else
    rms_norm_backward_kernel<X, S, 16, 4><<<p.grid, threads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t st) {
  if (a.bf16 && a.stream_bf16)
    return a.e4m3 ? pick_fwd<uint16_t, uint16_t, true>(a, st)
                  : pick_fwd<uint16_t, uint16_t, false>(a, st);
  if (a.bf16)
    return a.e4m3 ? pick_fwd<uint16_t, float, true>(a, st)
                  : pick_fwd<uint16_t, float, false>(a, st);
  return a.e4m3 ? pick_fwd<float, float, true>(a, st) : pick_fwd<float, float, false>(a, st);
}

size_t rms_norm_backward_partials(int64_t T, int d) {
  const GradPlan p = grad_plan(T, d);
  return size_t(p.grid) * p.rows;
}

hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t st) {
  const GradPlan p = grad_plan(a.T, a.d);
  hipError_t e = hipSuccess;
  if (a.T == 0)
    ;
  else if (a.bf16 && a.stream_bf16)
    e = run_bwd<uint16_t, uint16_t>(a, p, st);
  else if (a.bf16)
    e = run_bwd<uint16_t, float>(a, p, st);
  else
    e = run_bwd<float, float>(a, p, st);
  if (e != hipSuccess || !a.dweight) return e;
  rms_norm_dweight_kernel<<<(a.d + kSumCols - 1) / kSumCols, kSumCols * kSumSlices, 0, st>>>(
      a.partial, a.T == 0 ? 0 : p.grid * p.rows, a.d, a.dweight);
  return hipGetLastError();
}

}  // namespace fff
