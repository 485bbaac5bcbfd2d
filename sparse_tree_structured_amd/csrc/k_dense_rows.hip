// Elementwise part of the dense block's backward passes, column sums, and
// activation checkpoints in 8 bits.  All are bound by HBM at large sizes:
// 16384 x 8192 of the gated pair from 8-bit sums, with h and an 8-bit x read
// back, moves 1.44 GB in 293 us (4.9 TB/s; a large copy moves 4.8), h alone 0.8
// GB in 176; a checkpoint of 16384 x 2048 in bf16 takes 17.4 us (101 MB, 5.8
// TB/s) and 16381 x 2040 are read back in 18.6.
#include <type_traits>

#include "dense.hpp"
#include "launch_dense.hpp"

namespace fff {
namespace {

// Columns a lane has: one 16-byte access of the layer's type.
template <typename E> constexpr int kLaneCols = 16 / int(sizeof(E));

__host__ __device__ constexpr int there(int64_t left, int most) {
  return left < 0 ? 0 : left < most ? static_cast<int>(left) : most;
}

// V values kept for the backward pass, in the layer's type or in 8 bits.
template <typename E, int V>
struct Saved {
  Pack<E, V> same;
  Pack<uint8_t, V> codes;
  float scale;

  template <bool STREAM>
  __device__ __forceinline__ void load(const void* save, const float* scales, int group, size_t row,
                                       int col, int N, int n) {
    if (scales) {
      codes.template load<STREAM>(static_cast<const uint8_t*>(save) + row * N + col, n);
      // V divides the group, and col is a multiple of V: one scale a lane
      scale = n > 0 ? scales[row * ((N + group - 1) / group) + col / group] : 0.0f;
    } else {
      same.template load<STREAM>(static_cast<const E*>(save) + row * N + col, n);
    }
  }
  __device__ __forceinline__ void get(float (&v)[V], bool eight) const {
    if (eight) {
      unpack_e4m3(codes, v);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= scale;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = same.get(i);
    }
  }
};

// Workgroup `block` of `blocks` that read a checkpoint: a wavefront has an
// access of 64 lanes at a time.
template <typename E>
__device__ __forceinline__ void restore_rows(const Restore& r, int64_t block, int64_t blocks) {
  constexpr int V = kLaneCols<E>;
  const int lane = threadIdx.x & (kWave - 1);
  const int strips = (r.d + kWave * V - 1) / (kWave * V);
  for (int64_t u = block * 4 + threadIdx.x / kWave; u < r.T * strips; u += blocks * 4) {
    const size_t t = static_cast<size_t>(u / strips);
    const int col = (static_cast<int>(u % strips) * kWave + lane) * V;
    const int n = there(r.d - col, V);
    Saved<E, V> q;
    q.template load<false>(r.codes, r.scale, r.group ? r.group : r.d, t, col, r.d, n);
    float v[V];
    q.get(v, true);
    if (n > 0) packed<E, V>(v).store(static_cast<E*>(r.x) + t * r.ld + col, n);
  }
}

int grid_of(int64_t units) {
  const int64_t b = (units + 3) / 4;
  return static_cast<int>(b < (1 << 20) ? b : (1 << 20));
}

int restore_grid(const Restore& r, bool bf16) {
  const int cols = kWave * (bf16 ? 8 : 4);
  return grid_of(r.T * ((int64_t(r.d) + cols - 1) / cols));
}

// Rows of a strip: 64 (four wavefronts take every fourth), or fewer where that
// leaves compute units without work: 512 x 1024 in bf16 takes 4 us with 4
// rows and 20 with 64, most of it one row's load after the other.
int strip_rows(int64_t T, int64_t col_blocks) {
  const int64_t r = T * col_blocks / 1024 / 4 * 4;
  return r < 4 ? 4 : r < 64 ? static_cast<int>(r) : 64;
}
constexpr int64_t kMaxStrips = 1024;  // a workgroup takes more than one, then

// In bf16 da and an x that is read back are rounded to bf16 here, once, for
// they are the next products' operands: each moves a gradient by up to 2^-8 of
// its terms' sizes.  (dW in bf16 from 8 bits is off by 0.29 % of its size in all,
// 0.17 with its own rounding alone.  An operand in two bf16 parts would double
// the products' time, nine tenths of the pass.)
//
// da = dy act'(pre); of the gated pair dgate = dh up act'(gate) and dup = dh
// act(gate), h = act(gate) up.  A workgroup has 64 lanes of columns and a
// strip of rows; column sums are added over its rows in order, then over its
// wavefronts, and one partial sum a strip is left for sum_strips_kernel.
// The workgroups after those read x back.
template <typename E, bool GATED, int ACT>
__global__ __launch_bounds__(256) void act_backward_kernel(ActBackward a, int col_blocks,
                                                           int64_t strips, int strip) {
  constexpr int V = kLaneCols<E>;
  const int64_t act_blocks = col_blocks * strips;
  if (blockIdx.x >= act_blocks) {
    restore_rows<E>(a.x, blockIdx.x - act_blocks, gridDim.x - act_blocks);
    return;
  }
  __shared__ float sums[GATED ? 1 : 4][GATED ? 1 : kWave * V];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int64_t first = blockIdx.x / col_blocks;
  const int col = (blockIdx.x % col_blocks * kWave + lane) * V;
  const int n = there(a.N - col, V);
  float total[V] = {};
  bool odd = false;
  // (with planes a row's padding is zeros in them)
  const int n_plane = a.da_planes[0].at ? there(a.da_planes[0].ld - col, V) : 0;
  const int n_da = there(a.da_ld - col, V);
  auto store_da = [&](int which, float (&v)[V], size_t row) {
    if (!a.da || n_da <= 0) return;
    if (n < V) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < n ? v[i] : 0.0f;
    }
    packed<E, V>(v).store(
        static_cast<E*>(a.da) + (which * static_cast<size_t>(a.T) + row) * a.da_ld + col, n_da);
  };
  auto planes = [&](int which, const float (&v)[V], size_t row) {
    if constexpr (sizeof(E) == 4)
      if (n_plane > 0)
        odd |= store_planes<V>(v, static_cast<uint16_t*>(a.da_planes[which].at) +
                                      row * a.da_planes[0].ld + col, a.da_planes[0].plane, n_plane);
  };
  for (int64_t r0 = first * strip; r0 < a.T; r0 += strips * strip) {
    const int64_t end = r0 + strip < a.T ? r0 + strip : a.T;
    for (int64_t t = r0 + wave; t < end; t += 4) {
      const size_t row = static_cast<size_t>(t);
      Pack<E, V> dy;
      Saved<E, V> pre, up;
      dy.template load<GATED>(static_cast<const E*>(a.dy) + row * a.N + col, n);
      if (a.save[0]) pre.template load<GATED>(a.save[0], a.scale[0], a.group, row, col, a.N, n);
      if constexpr (GATED) up.template load<true>(a.save[1], a.scale[1], a.group, row, col, a.N, n);
      float p[V], da[V];
      if (a.save[0]) pre.get(p, a.scale[0] != nullptr);
      if constexpr (GATED) {
        float w[V], du[V], h[V];
        up.get(w, a.scale[1] != nullptr);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float value, slope;
          activation_slope(p[i], ACT, value, slope);
          da[i] = dy.get(i) * w[i] * slope;
          du[i] = dy.get(i) * value;
          h[i] = value * w[i];
        }
        planes(0, da, row);
        planes(1, du, row);
        store_da(0, da, row);
        store_da(1, du, row);
        if (a.h && n > 0)
          packed<E, V>(h).template store<true>(static_cast<E*>(a.h) + row * a.N + col, n);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          da[i] = dy.get(i);
          if (a.save[0]) {
            float value, slope;
            activation_slope(p[i], ACT, value, slope);
            da[i] *= slope;
          }
          total[i] += da[i];
        }
        planes(0, da, row);
        store_da(0, da, row);
      }
    }
  }
  if (odd) *a.bad.word = a.bad.call;
  if constexpr (!GATED) {
    if (!a.partial) return;
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][lane * V + i] = total[i];
    __syncthreads();
    for (int c = threadIdx.x; c < kWave * V; c += 256) {
      const int at = blockIdx.x % col_blocks * kWave * V + c;
      if (at < a.N)
        a.partial[static_cast<size_t>(first) * a.N + at] =
            (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
    }
  }
}

// dbias from the strips' sums: 16 columns to a workgroup, 16 threads each.
__global__ __launch_bounds__(256) void sum_strips_kernel(const float* partial, int strips, int N,
                                                         float* out) {
  __shared__ float lds[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;
  float s = 0.0f;
  if (col < N)
    for (int i = r; i < strips; i += 16) s += partial[static_cast<size_t>(i) * N + col];
  lds[r][c] = s;
  __syncthreads();
  if (r == 0 && col < N) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += lds[i][c];
    out[col] = s;
  }
}

// ---- checkpoints ----

// A wavefront a row: with groups, scales come from the lanes of a group; with
// one scale a row, the row is read twice (the second time from cache).
template <typename E>
__global__ __launch_bounds__(256) void checkpoint_save_kernel(int64_t T, int d, int group, const E* x,
                                                              uint8_t* codes, float* scale) {
  constexpr int V = kLaneCols<E>;
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t t = int64_t(blockIdx.x) * 4 + threadIdx.x / kWave; t < T; t += int64_t(gridDim.x) * 4) {
    const E* row = x + static_cast<size_t>(t) * d;
    uint32_t top = 0;
    if (group == 0) {
      for (int c0 = 0; c0 < d; c0 += kWave * V) {
        const int col = c0 + lane * V;
        Pack<E, V> p;
        p.load(row + col, there(d - col, V));
#pragma unroll
        for (int i = 0; i < V; ++i) top = umax(top, size_bits(p.get(i)));
      }
      top = wave_max(top);
      if (lane == 0) scale[t] = e4m3_scale(top);
    }
    const float inv = reciprocal(e4m3_scale(top));
    for (int c0 = 0; c0 < d; c0 += kWave * V) {
      const int col = c0 + lane * V;
      const int n = there(d - col, V);
      Pack<E, V> p;
      p.load(row + col, n);
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = p.get(i);
      if (group != 0) {
        save_e4m3(v, n, codes, scale, t, col, d, group);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= inv;
        pack_e4m3(v).store(codes + static_cast<size_t>(t) * d + col, n);
      }
    }
  }
}

template <typename E>
__global__ __launch_bounds__(256) void checkpoint_load_kernel(Restore r) {
  restore_rows<E>(r, blockIdx.x, gridDim.x);
}

int64_t col_blocks_of(int N, bool bf16) {
  const int cols = kWave * (bf16 ? 8 : 4);
  return (int64_t(N) + cols - 1) / cols;
}

int64_t strips_of(int64_t T, int N, bool bf16) {
  const int r = strip_rows(T, col_blocks_of(N, bf16));
  const int64_t s = (T + r - 1) / r;
  return s < kMaxStrips ? s : kMaxStrips;
}

template <typename E, bool GATED>
hipError_t run_act_backward(ActBackward a, hipStream_t st) {
  constexpr bool kBf16 = sizeof(E) == 2;
  const int64_t col_blocks = col_blocks_of(a.N, kBf16);
  // (nothing to do for dy's columns: x alone)
  const int64_t strips = a.da || a.h || a.dbias ? strips_of(a.T, a.N, kBf16) : 0;
  const int64_t blocks = col_blocks * strips + (a.x.x ? restore_grid(a.x, kBf16) : 0);
  const bool one_strip = strips == 1 && a.dbias;  // its sums are the result
  if (one_strip) a.partial = a.dbias;
  if (blocks > 0) {
    auto launch = [&](auto act) {
      act_backward_kernel<E, GATED, decltype(act)::value>
          <<<dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, st>>>(
              a, static_cast<int>(col_blocks), strips, strip_rows(a.T, col_blocks));
    };
    switch (a.act) {
      case kActGelu: launch(std::integral_constant<int, kActGelu>()); break;
      case kActSilu: launch(std::integral_constant<int, kActSilu>()); break;
      case kActRelu: launch(std::integral_constant<int, kActRelu>()); break;
      default: launch(std::integral_constant<int, kActNone>());
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dbias && !one_strip) {
    sum_strips_kernel<<<dim3((a.N + 15) / 16), dim3(256), 0, st>>>(a.partial, static_cast<int>(strips),
                                                                   a.N, a.dbias);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

size_t act_backward_partials(int64_t T, int N, bool bf16) {
  return size_t(strips_of(T, N, bf16)) * size_t(N);
}

hipError_t launch_act_backward(const ActBackward& a, hipStream_t st) {
  if (a.gated)
    return a.bf16 ? run_act_backward<uint16_t, true>(a, st) : run_act_backward<float, true>(a, st);
  return a.bf16 ? run_act_backward<uint16_t, false>(a, st) : run_act_backward<float, false>(a, st);
}

hipError_t launch_checkpoint_save(int64_t T, int d, bool bf16, int group, const void* x, void* codes,
                                  float* scale, hipStream_t st) {
  uint8_t* q = static_cast<uint8_t*>(codes);
  if (bf16)
    checkpoint_save_kernel<uint16_t><<<grid_of(T), 256, 0, st>>>(
        T, d, group, static_cast<const uint16_t*>(x), q, scale);
  else
    checkpoint_save_kernel<float><<<grid_of(T), 256, 0, st>>>(T, d, group,
                                                              static_cast<const float*>(x), q, scale);
  return hipGetLastError();
}

hipError_t launch_checkpoint_load(int64_t T, int d, bool bf16, int group, const void* codes,
                                  const float* scale, void* x, hipStream_t st) {
  const Restore r = {T, d, group, codes, scale, x, d};
  const int grid = restore_grid(r, bf16);
  if (bf16)
    checkpoint_load_kernel<uint16_t><<<grid, 256, 0, st>>>(r);
  else
    checkpoint_load_kernel<float><<<grid, 256, 0, st>>>(r);
  return hipGetLastError();
}

}  // namespace fff
