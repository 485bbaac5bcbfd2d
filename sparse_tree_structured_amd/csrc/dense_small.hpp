// Products x . W of few rows (a decode step): the weights are read once,
// straight into registers, and nothing else takes time.
//
// A workgroup has 64 output columns and a slice of K; its eight wavefronts
// take every eighth 32 rows of W (of a gated pair, of both).  A lane loads four columns of eight rows, so that 16
// lanes have whole lines, and has then, for each of its columns, eight
// consecutive k: after a 16-bit transpose in its registers (one byte permute
// for two values) that is an operand of v_mfma_f32_16x16x32_bf16, with x's
// rows as the other; float32 uses v_mfma_f32_16x16x4_f32 on the values as
// they are.  Several steps' loads are in flight.
//
// The wavefronts' sums are added through LDS in their order.  Where K is cut,
// a slice's sums go to the workspace past the caches of one XCD, and the
// workgroup that finds all slices of its columns there adds them in their
// order and writes the output: one launch, and the same result on every call.
// Bound by HBM and, for the smallest, by launch and latency: one token through
// a bf16 pair of 2048 x 8192 reads 67 MB in 14.7 us a call (4.6 TB/s; a large
// copy moves 4.8), 64 tokens take 19.6 (x's rows come from L2 in every
// workgroup); 1 x 8192 x 2048 takes 8.3 us on the GPU, 10.9 a call.
// (Counting arrivals with compare and exchange took 20 us of 35 where 16
// slices meet; a second launch takes 4 us of the host's time.)
#pragma once

#include <type_traits>

#include "dense.hpp"

namespace fff {

constexpr int kSmallRows = 64;     // most rows
constexpr int kSmallCols = 64;     // of a workgroup
constexpr int kSmallWaves = 8;
constexpr int kSmallStep = 32;     // of K
constexpr int kSmallMaxSlices = 64;

// Arrivals at a column block.  Each slice writes the call's number into a
// word of its own and then looks at all of them; who sees them all has the
// sums in memory, and the first of those to exchange the last word finishes.
// Numbers are unique, so nothing has to be cleared: what other calls left, or
// what was in the memory before, is none.  (A captured call's number would be
// there from the replay before: its sums take a second launch.)
struct SmallArrival {
  unsigned long long call;    // 0: a second launch adds the slices
  unsigned long long* words;  // [block][slices + 1]
};

// For one wavefront.
__device__ __forceinline__ bool finishes(const SmallArrival& a, int block, int slice, int slices,
                                         int lane) {
  unsigned long long* w = a.words + static_cast<size_t>(block) * (slices + 1);
  if (lane == 0) __hip_atomic_store(w + slice, a.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  asm volatile("" ::: "memory");
  wait_vmcnt<0>();  // it is in memory
  asm volatile("" ::: "memory");
  unsigned long long there = a.call;
  if (lane < slices) there = __hip_atomic_load(w + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (__ballot(there != a.call) != 0) return false;
  unsigned long long before = a.call;
  if (lane == 0)
    before = __hip_atomic_exchange(w + slices, a.call, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __ballot(before != a.call) != 0;
}

constexpr int kDeviceScope = 16;  // buffer cache policy: sc1
__device__ __forceinline__ __amdgpu_buffer_rsrc_t part_buffer(float* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(p, 0, bytes, 0x00020000);
}

// One step's operands of a lane.
template <typename E, int TT, int W>
struct SmallStep {
  Pack<E, 4> w[W][8];
  Pack<E, 16 / int(sizeof(E))> x[TT][sizeof(E) / 2];  // eight values of each row

  __device__ __forceinline__ void load(const E* x_at, int64_t ldx, int T, const E* const (&w_at)[W],
                                       int64_t ldw, int k0, int K, int cols, int lane) {
    constexpr int V = 16 / int(sizeof(E));
    const int k = k0 + (lane >> 4) * 8;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (k0 + kSmallStep <= K) {
#pragma unroll
        for (int r = 0; r < 8; ++r) w[i][r].load(w_at[i] + (k + r) * ldw, cols);
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r) w[i][r].load(w_at[i] + (k + r) * ldw, k + r < K ? cols : 0);
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int row = t * 16 + (lane & 15);
      const E* p = x_at + (row < T ? row : T - 1) * ldx + k;
#pragma unroll
      for (int h = 0; h < int(sizeof(E)) / 2; ++h) x[t][h].load(p + h * V, K - k - h * V);
    }
  }
};

typedef float f32x4_t __attribute__((ext_vector_type(4)));

template <typename E, int TT, int W>
__device__ __forceinline__ void small_mma(f32x4_t (&acc)[W][4][TT], const SmallStep<E, TT, W>& s) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (sizeof(E) == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 f;
        uint32_t* d = &f.x;
#pragma unroll
        for (int r = 0; r < 4; ++r)  // rows 2 r and 2 r + 1 of column j
          d[r] = __builtin_amdgcn_perm(s.w[i][2 * r + 1].word(j >> 1), s.w[i][2 * r].word(j >> 1),
                                       j & 1 ? 0x07060302u : 0x05040100u);
        const bf16x8_t wf = __builtin_bit_cast(bf16x8_t, f);
#pragma unroll
        for (int t = 0; t < TT; ++t)
          acc[i][j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, s.x[t][0].q), wf, acc[i][j][t], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)  // a lane's k = 8 (lane / 16) + r
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < TT; ++t)
            acc[i][j][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                s.x[t][r / 4].get(r % 4), s.w[i][r].get(j), acc[i][j][t], 0, 0, 0);
    }
  }
}

// Row `row` of a column block: the slices' sums [slice][v, w][ROWS][column]
// in their order, and the epilogue.
template <int ROWS, class Epi>
__device__ __forceinline__ void add_slices(const Epi& epi, const typename Epi::Column& column,
                                           __amdgpu_buffer_rsrc_t buf, int row, int col, int n, int c4,
                                           int slices) {
  constexpr int kOne = ROWS * kSmallCols;
  typename Epi::Early early;
  epi.early(early, row, col, n);
  float v[4] = {}, g[4] = {};
  auto part = [&](uint32_t at) {
    return __builtin_bit_cast(float4,
                              __builtin_amdgcn_raw_buffer_load_b128(buf, at * 4, 0, kDeviceScope));
  };
  auto add = [](float (&to)[4], const float4& q) {
    to[0] += q.x; to[1] += q.y; to[2] += q.z; to[3] += q.w;
  };
  constexpr int kBatch = 8;  // loads on their way together
  for (int i = 0; i < slices; i += kBatch) {
    float4 q[kBatch], r[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k < slices) {
        const uint32_t at = uint32_t(i + k) * (Epi::kGated ? 2 : 1) * kOne + row * kSmallCols + c4;
        q[k] = part(at);
        if constexpr (Epi::kGated) r[k] = part(at + kOne);
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k < slices) {
        add(v, q[k]);
        if constexpr (Epi::kGated) add(g, r[k]);
      }
  }
  epi.apply(column, early, row, col, n, v, g, 0);
}

template <int TT>
constexpr size_t small_lds() { return size_t(kSmallWaves) * TT * 16 * kSmallCols * sizeof(float); }

template <typename E, int TT, class Epi>
__global__ __launch_bounds__(kSmallWaves * kWave) void product_small_kernel(Product p, Epi epi,
                                                                            int col_blocks, int slices,
                                                                            int steps, float* partial,
                                                                            SmallArrival arrival) {
  constexpr bool G = Epi::kGated;
  constexpr int kRows = TT * 16;
  constexpr int W = G ? 2 : 1;
  // Steps in flight: as many as the registers hold.
  constexpr int kStepRegs = (W * 16 + TT * 4) * int(sizeof(E)) / 2;
  constexpr int kDepth = kStepRegs <= 28 ? 4 : kStepRegs <= 64 ? 2 : 1;
  extern __shared__ __align__(16) float sums[];  // [wave][row][column]
  __shared__ int last;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int block = blockIdx.x % col_blocks;
  const int slice = blockIdx.x / col_blocks;
  const int n0 = block * kSmallCols;
  const int T = static_cast<int>(p.M), K = static_cast<int>(p.K);
  const int col = n0 + (lane & 15) * 4;
  const int cols = p.N - col < 4 ? p.N - col : 4;  // (none: not above 0)
  const E* x = static_cast<const E*>(p.a);
  const E* w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = static_cast<const E*>(p.b[i]) + col;
  const int total = (K + kSmallStep - 1) / kSmallStep;
  const int end = (slice + 1) * steps < total ? (slice + 1) * steps : total;
  f32x4_t acc[W][4][TT];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[i][j][t] = f32x4_t{};
  SmallStep<E, TT, W> s[kDepth];
  int at = slice * steps + wave;
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (at + d * kSmallWaves < end)
      s[d].load(x, p.lda, T, w, p.ldb, (at + d * kSmallWaves) * kSmallStep, K, cols, lane);
  for (; at < end; at += kDepth * kSmallWaves) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int now = at + d * kSmallWaves;
      if (now < end) {
        small_mma<E, TT, W>(acc, s[d]);
        const int next = now + kDepth * kSmallWaves;
        if (next < end)
          s[d].load(x, p.lda, T, w, p.ldb, next * kSmallStep, K, cols, lane);
      }
    }
  }
  constexpr int kUnits = kRows * kSmallCols / 4;  // four columns of a row
  const int c4 = (tid & 15) * 4;
  const int left = p.N - (n0 + c4);
  const int n_col = left < 0 ? 0 : left < 4 ? left : 4;
  auto add = [](float (&v)[4], const float4& q) {
    v[0] += q.x; v[1] += q.y; v[2] += q.z; v[3] += q.w;
  };
  typename Epi::Column column;
  epi.column(column, n0 + c4);
  // One slice's sums of a block: [slice][v, w][row][column].
  constexpr int kPart = W * kRows * kSmallCols;
  float* const parts = partial + static_cast<size_t>(block) * slices * kPart;
  const __amdgpu_buffer_rsrc_t buf = part_buffer(parts, uint32_t(slices) * kPart * 4);
  // The wavefronts' sums of one weight after the other's.
  constexpr int kThreads = kSmallWaves * kWave;
  constexpr int kMine = (kUnits + kThreads - 1) / kThreads;
  float v[W][kMine][4] = {};
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i > 0) __syncthreads();
    // acc[i][j][t][r]: row 16 t + 4 (lane / 16) + r, column 4 (lane % 16) + j.
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4*>(sums + (wave * kRows + t * 16 + (lane >> 4) * 4 + r) * kSmallCols +
                                   (lane & 15) * 4) =
            make_float4(acc[i][0][t][r], acc[i][1][t][r], acc[i][2][t][r], acc[i][3][t][r]);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int row = (tid + m * kThreads) >> 4;
      if (row < kRows)
#pragma unroll
        for (int k = 0; k < kSmallWaves; ++k)
          add(v[i][m], *reinterpret_cast<const float4*>(sums + (k * kRows + row) * kSmallCols + c4));
    }
  }
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int row = (tid + m * kThreads) >> 4;
    if (row >= kRows) break;
    if (slices == 1) {
      typename Epi::Early early;
      const int n = row < T ? n_col : 0;
      epi.early(early, row, n0 + c4, n);
      epi.apply(column, early, row, n0 + c4, n, v[0][m], v[W - 1][m], 0);
    } else if (row < T) {
      typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
#pragma unroll
      for (int i = 0; i < W; ++i)
        __builtin_amdgcn_raw_buffer_store_b128(
            __builtin_bit_cast(u32x4_t, make_float4(v[i][m][0], v[i][m][1], v[i][m][2], v[i][m][3])), buf,
            (uint32_t(slice) * kPart + i * kRows * kSmallCols + row * kSmallCols + c4) * 4, 0,
            kDeviceScope);
    }
  }
  if (slices == 1 || arrival.call == 0) return;
  // Every wavefront's sums are in memory before the workgroup arrives.
  asm volatile("" ::: "memory");
  wait_vmcnt<0>();
  __syncthreads();
  if (wave == 0) {
    const bool mine = finishes(arrival, block, slice, slices, lane);
    if (lane == 0) last = mine;
  }
  __syncthreads();
  if (!last) return;
  for (int u = tid; u < T * 16; u += kSmallWaves * kWave)
    add_slices<kRows>(epi, column, buf, u >> 4, n0 + c4, n_col, c4, slices);
}

// The same where the slices' sums were left to a second launch: one workgroup
// to a column block.
template <int TT, class Epi>
__global__ __launch_bounds__(kSmallWaves * kWave) void small_slices_kernel(Epi epi, int T, int N,
                                                                           int slices, float* partial) {
  constexpr int kPart = (Epi::kGated ? 2 : 1) * TT * 16 * kSmallCols;
  const int c4 = (threadIdx.x & 15) * 4;
  const int col = blockIdx.x * kSmallCols + c4;
  const int left = N - col;
  const __amdgpu_buffer_rsrc_t buf =
      part_buffer(partial + static_cast<size_t>(blockIdx.x) * slices * kPart, uint32_t(slices) * kPart * 4);
  typename Epi::Column column;
  epi.column(column, col);
  for (int u = threadIdx.x; u < T * 16; u += kSmallWaves * kWave)
    add_slices<TT * 16>(epi, column, buf, u >> 4, col, left < 0 ? 0 : left < 4 ? left : 4, c4, slices);
}

}  // namespace fff
