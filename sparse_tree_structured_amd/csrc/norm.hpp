// What the norm's kernels share: rows held in the registers of a team of
// wavefronts.
#pragma once

#include "common.hpp"
#include "launch_train.hpp"
#include "train.hpp"

namespace fff {

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
  template <bool STREAM = false, typename E>
  __device__ __forceinline__ void store(const Pack<E, V>& p, E* row) const {
    if (in) p.template store<STREAM>(row + first, V);
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
// 8000 x 2703 in bf16 the forward takes 41.1 us instead of 53.6); what the
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
  template <bool STREAM = false, typename E>
  __device__ __forceinline__ void store(const Pack<E, V>& p, E* row) const {
    if (lo == 0 && hi == V)
      p.template store<STREAM>(row + col, V);
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

// Wavefronts of a row and chunks of each.
struct RowPlan {
  int waves, chunks;
  int rows() const { return waves == 1 ? 4 : 1; }  // of a workgroup
  int threads() const { return block_threads(waves); }
};

// Accesses of one wavefront that a row takes: at most 128, or 64 of eight
// columns a lane.
inline int pieces_of(int d, int cols) { return (d + cols * kWave - 1) / (cols * kWave); }

template <int W, int C> struct Plan {
  static constexpr int kWaves = W, kChunks = C;
};

}  // namespace fff
