// Epilogues of the bf16 products on the accumulators as they lie in the
// registers: a lane has a row and, of each 32 columns, 8 g + 4 (lane / 32) +
// 0..3.  Biases, activations and 8-bit scales are formed there and the
// outputs go through LDS in the form in which they are written, once for the
// tile, so that every store is 16 bytes a lane in whole lines.
//
// tile_epilogue (dense.hpp) takes 32-bit sums through LDS in bands and does
// four columns a lane at a time: at 16384 x 2048 x 8192 its 8-bit saves cost
// 257 us of 1239 (five steps over lanes and a scale for every four columns;
// here one step and a scale for 16; 1056 in all), and at 16384 x 2048 x 16384
// its plain outputs 160 us of 1040 (here 60).  A linear layer whose sums are
// kept, or whose output is in 32 bits, and products on planes still take it:
// 16384 x 2048 x 8192 with bias and GELU takes 541 us, and keeping its sums 627
// (in the layer's type) or 677 (in 8 bits); without them but with a 32-bit
// residual and output 658.
#pragma once

#include "dense.hpp"

namespace fff {

// 16-byte pieces of a staged tile (rows of PITCH bytes, COLS columns of E) to
// an output of N columns.
template <typename E, int ROWS, int COLS, int PITCH, int THREADS>
__device__ __forceinline__ void store_staged(const unsigned char* stage, E* out, int64_t m0, int64_t M,
                                             int n0, int N) {
  constexpr int V = 16 / sizeof(E);
  constexpr int kPieces = COLS / V;
  static_assert(ROWS * kPieces % THREADS == 0, "pieces split evenly");
#pragma unroll
  for (int i = 0; i < ROWS * kPieces / THREADS; ++i) {
    const int p = threadIdx.x + i * THREADS;
    const int r = p / kPieces, c = p % kPieces * V;
    const int64_t row = m0 + r;
    const int left = N - (n0 + c);
    if (row >= M || left <= 0) continue;
    Pack<E, V> v;
    v.q = *reinterpret_cast<const decltype(v.q)*>(stage + r * PITCH + c * sizeof(E));
    v.store(out + static_cast<size_t>(row) * N + n0 + c, left);
  }
}

template <int ACT>
__device__ __forceinline__ float activation_of(float a) { return activation(a, ACT); }

// f with the activation as a constant.
template <class F>
__device__ __forceinline__ void with_activation(int act, const F& f) {
  switch (act) {
    case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
    default: f(std::integral_constant<int, kActNone>());
  }
}

// ---- the gated pair: acc[i][0] is of x . W_gate, acc[i][1] of x . W_up ----

template <class C>
struct GatedStage {
  static constexpr int kCols = C::BN / 2;        // 128
  static constexpr int kPitch = kCols * 2 + 16;  // bytes of a bf16 row
  static constexpr int kCodePitch = kCols + 16;
  static constexpr int kTile = C::BM * kPitch;
  static constexpr int kCodes = C::BM * kCodePitch;
  static constexpr int kTops = 2 * C::BM * 16;  // largest sizes by row and wavefront column
  static constexpr size_t kEights = kTile + 2 * kCodes + kTops;
  static constexpr size_t kSame = 2 * kTile;
  static constexpr size_t kBytes = kEights > kSame ? kEights : kSame;
  static_assert(C::WN == 64 && C::kTn == 2 && C::kWavesN == 4, "a wavefront has 32 columns of each");
};

template <class C>
__device__ __forceinline__ void gated_epilogue(const f32x16_t (&acc)[C::kTm][C::kTn],
                                               unsigned char* lds, const Epilogue& e, int64_t m0,
                                               int n0) {
  using S = GatedStage<C>;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int wm = wave / C::kWavesN, wn = wave % C::kWavesN;
  const int hi = lane >> 5;
  const int row0 = wm * C::WM + (lane & 31);  // of the tile, and + 32 i
  const int col0 = wn * 32 + hi * 4;          // of the tile, and + 8 g
  auto stage_bf16 = [&](unsigned char* at, int i, const float (&v)[16]) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<uint2*>(at + (row0 + i * 32) * S::kPitch + (col0 + g * 8) * 2) =
          make_uint2(pack_bf16x2(v[4 * g], v[4 * g + 1]), pack_bf16x2(v[4 * g + 2], v[4 * g + 3]));
  };
  auto sums_of = [&](int i, int j, float (&v)[16]) {
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = acc[i][j][r];
  };
  unsigned char* const h_at = lds;
  unsigned char* const code_at = lds + S::kTile;
  uint32_t* const tops = reinterpret_cast<uint32_t*>(lds + S::kTile + 2 * S::kCodes);
  const bool edge = n0 + S::kCols > e.N;
  with_activation(e.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < C::kTm; ++i) {
      float h[16];
#pragma unroll
      for (int r = 0; r < 16; ++r)
        h[r] = activation_of<decltype(act)::value>(acc[i][0][r]) * acc[i][1][r];
      stage_bf16(h_at, i, h);
    }
  });
  bool eights[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    eights[w] = e.save[w] && e.scale[w];
    if (eights[w]) {
#pragma unroll
      for (int i = 0; i < C::kTm; ++i) {
        uint32_t top = 0;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          uint32_t b = size_bits(acc[i][w][r]);
          // (columns past the end are of other columns' values)
          if (edge && n0 + col0 + (r / 4) * 8 + r % 4 >= e.N) b = 0;
          top = umax(top, b);
        }
        const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
        if (hi == 0) tops[(w * C::BM + row0 + i * 32) * 4 + wn] = umax(both[0], both[1]);
      }
    }
  }
  // In the layer's type: the gate's sums beside h, the other's after them.
  const bool same0 = e.save[0] && !e.scale[0], same1 = e.save[1] && !e.scale[1];
  if (same0) {
#pragma unroll
    for (int i = 0; i < C::kTm; ++i) {
      float v[16];
      sums_of(i, 0, v);
      stage_bf16(lds + S::kTile, i, v);
    }
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (!eights[w]) continue;
#pragma unroll
    for (int i = 0; i < C::kTm; ++i) {
      const int r = row0 + i * 32;
      const uint4 t = *reinterpret_cast<const uint4*>(tops + (w * C::BM + r) * 4);
      const uint32_t lo = umax(t.x, t.y), up = umax(t.z, t.w);
      const uint32_t top = e.group == 128  ? umax(lo, up)
                           : e.group == 64 ? (wn < 2 ? lo : up)
                                           : (wn < 2 ? (wn ? t.y : t.x) : (wn == 3 ? t.w : t.z));
      const float scale = e4m3_scale(top);
      const float inv = reciprocal(scale);
      float q[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) q[k] = acc[i][w][k] * inv;
      const Pack<uint8_t, 16> codes = pack_e4m3(q);
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<uint32_t*>(code_at + w * S::kCodes + r * S::kCodePitch + col0 + g * 8) =
            codes.word(g);
      const int col = n0 + wn * 32;
      if (hi == 0 && col % e.group == 0 && m0 + r < e.M && col < e.N)
        e.scale[w][static_cast<size_t>(m0 + r) * ((e.N + e.group - 1) / e.group) + col / e.group] =
            scale;
    }
  }
  if (eights[0] || eights[1]) __syncthreads();
  store_staged<uint16_t, C::BM, S::kCols, S::kPitch, C::kThreads>(
      h_at, static_cast<uint16_t*>(e.out[0]), m0, e.M, n0, e.N);
#pragma unroll
  for (int w = 0; w < 2; ++w)
    if (eights[w])
      store_staged<uint8_t, C::BM, S::kCols, S::kCodePitch, C::kThreads>(
          code_at + w * S::kCodes, static_cast<uint8_t*>(e.save[w]), m0, e.M, n0, e.N);
  if (same0)
    store_staged<uint16_t, C::BM, S::kCols, S::kPitch, C::kThreads>(
        lds + S::kTile, static_cast<uint16_t*>(e.save[0]), m0, e.M, n0, e.N);
  if (same1) {
    __syncthreads();  // h has been read
#pragma unroll
    for (int i = 0; i < C::kTm; ++i) {
      float v[16];
      sums_of(i, 1, v);
      stage_bf16(h_at, i, v);
    }
    __syncthreads();
    store_staged<uint16_t, C::BM, S::kCols, S::kPitch, C::kThreads>(
        h_at, static_cast<uint16_t*>(e.save[1]), m0, e.M, n0, e.N);
  }
}

// ---- a linear layer whose output is bf16 and whose sums are not kept ----

// The staged tile: rows of BN columns, 16-byte piece c of row r at slot
// c ^ (r mod kPieces), so that 32 rows' accesses to one column spread over the
// banks without padding, which copies straight into LDS could not make.
template <class C>
struct LinearStage {
  static constexpr int kPieces = C::BN / 8;
  static constexpr int kPitch = C::BN * 2;
  static constexpr size_t kBytes = size_t(C::BM) * kPitch;
  static __device__ __forceinline__ int slot(int row, int piece) {
    return row * kPitch + ((piece ^ (row & (kPieces - 1))) << 4);
  }
};

// Needs a residual of 16-byte alignment.
template <class C>
__device__ __forceinline__ void linear_epilogue(const f32x16_t (&acc)[C::kTm][C::kTn], unsigned char* lds,
                                                const Epilogue& e, int64_t m0, int n0, int which) {
  using S = LinearStage<C>;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int wm = wave / C::kWavesN, wn = wave % C::kWavesN;
  const int row0 = wm * C::WM + (lane & 31);
  const int col0 = wn * C::WN + (lane >> 5) * 4;
  // The residual to where y will be staged, on its way while the activations
  // are formed.  What is past its end comes from its last row or the tile's
  // first columns, and is not written.
  if (e.residual) {
    constexpr int kCopies = C::BM * S::kPitch / 1024 / C::kWaves;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int q = (wave * kCopies + i) * 1024;
      const int r = (q + lane * 16) / S::kPitch;
      const int c = ((lane % S::kPieces) ^ (r & (S::kPieces - 1))) * 8;
      const int64_t row = m0 + r < e.M ? m0 + r : e.M - 1;
      const int col = n0 + c < e.N ? n0 + c : n0;
      dma16_asm(static_cast<const uint16_t*>(e.residual) + static_cast<size_t>(row) * e.N + col,
                lds + q);
    }
  }
  float bias[C::kTn][16];
#pragma unroll
  for (int j = 0; j < C::kTn; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = n0 + col0 + j * 32 + g * 8;
      Pack<uint16_t, 4> b = {};
      if (e.bias) b.load(static_cast<const uint16_t*>(e.bias) + col, e.N - col);
#pragma unroll
      for (int k = 0; k < 4; ++k) bias[j][4 * g + k] = b.get(k);
    }
  if (e.residual) {
    wait_vmcnt<0>();
    stage_barrier();
  }
#pragma unroll
  for (int i = 0; i < C::kTm; ++i) {
    float v[C::kTn][16];
#pragma unroll
    for (int j = 0; j < C::kTn; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) v[j][k] = acc[i][j][k] + bias[j][k];
    if (e.act != kActNone)
      with_activation(e.act, [&](auto act) {
#pragma unroll
        for (int j = 0; j < C::kTn; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) v[j][k] = activation_of<decltype(act)::value>(v[j][k]);
      });
#pragma unroll
    for (int j = 0; j < C::kTn; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = col0 + j * 32 + g * 8;
        uint2* at = reinterpret_cast<uint2*>(lds + S::slot(row0 + i * 32, c >> 3) + (c & 7) * 2);
        float* y = v[j] + 4 * g;
        if (e.residual) {
          const uint2 w = *at;
          y[0] += bf16lo(w.x);
          y[1] += bf16hi(w.x);
          y[2] += bf16lo(w.y);
          y[3] += bf16hi(w.y);
        }
        *at = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      }
  }
  __syncthreads();
  uint16_t* out = static_cast<uint16_t*>(e.out[which]);
#pragma unroll
  for (int i = 0; i < C::BM * S::kPieces / C::kThreads; ++i) {
    const int p = threadIdx.x + i * C::kThreads;
    const int r = p / S::kPieces, c = p % S::kPieces;
    const int left = e.N - (n0 + c * 8);
    if (m0 + r >= e.M || left <= 0) continue;
    Pack<uint16_t, 8> v;
    v.q = *reinterpret_cast<const decltype(v.q)*>(lds + S::slot(r, c));
    v.store(out + static_cast<size_t>(m0 + r) * e.N + n0 + c * 8, left);
  }
}

}  // namespace fff
