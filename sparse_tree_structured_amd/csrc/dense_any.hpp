// Register-staged product of any sizes and alignment, float32 or bf16.
//
// Operands go from memory into registers a K step ahead of their use, as
// 16-byte accesses of one element's alignment (short at the ends of rows, so
// nothing outside a tensor is read and what is not there is zero), and from
// there into two LDS buffers.  bf16 uses v_mfma_f32_32x32x16_bf16 on the
// layouts of mfma_tile.hpp; float32 v_mfma_f32_32x32x2_f32, whose products
// and sums are those of 32-bit arithmetic.
//
// Float32 is bound by its matrix operations (a compute unit's 128 x 256 x 16
// step takes 1.9 us at full rate): 16384 x 8192 x 2048 runs at 120 TFLOP/s.
// bf16 steps of 32 take 0.75 to 0.8 us, most of it addresses and guards, where
// rows are whole 16-byte pieces at odd addresses (16384 x 8192 x 2048 814 us, 0.68
// PFLOP/s; 483 aligned, straight into LDS), and 0.7 to 1.3 us with odd rows (16384
// x 2047 x 8191 743 us, 4096 x 4095 x 4095 327; 513 and 137 with copies, straight
// into LDS): bf16 comes here where pointers are not aligned, or rows are odd and
// copies are not worth their time.  Two steps' loads in registers changed nothing.
#pragma once

#include "dense.hpp"

namespace fff {

enum Layout { kRows, kKMajor };  // of an operand: K contiguous, or k-major

// OUTER rows (or columns) of an operand by BK of K.
template <typename E, int OUTER, int BK, Layout L, int THREADS>
struct Stager {
  static constexpr int V = 16 / sizeof(E);
  static constexpr int kPer = L == kRows ? BK / V : OUTER / V;  // accesses of a row
  static constexpr int kChunks = OUTER * BK / V / THREADS;
  static_assert(OUTER * BK / V % THREADS == 0, "accesses split evenly");
  // LDS: bf16 as mfma_tile.hpp has it; float32 rows of BK + 4, or k rows of
  // OUTER + 8, which keep the operand reads below free of bank conflicts.
  static constexpr int kPitch = sizeof(E) == 2 ? (L == kRows ? BK : OUTER)
                                               : (L == kRows ? BK + 4 : OUTER + 8);
  static constexpr int kBytes = (L == kRows ? OUTER : BK) * kPitch * int(sizeof(E));
  static_assert(sizeof(E) == 4 || L == kRows || OUTER % 128 == 0, "swizzle spans 16 chunks");
  Pack<E, V> r[kChunks];

  // (rows of 128 bytes have eight chunks: 16 rows' reads of one chunk cover
  // all banks with the row's bits 1 to 3, as with bits 2 and 3 for 64 bytes)
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (L == kKMajor) return (row & 3) << 2;
    return BK == 64 ? (row >> 1) & 7 : lds_swz(row);
  }
  static __device__ __forceinline__ int slot(int row, int chunk) {
    if constexpr (sizeof(E) == 2) chunk ^= swizzle(row);
    return (row * kPitch + chunk * V) * int(sizeof(E));
  }
  // p: element (first row or column, k = 0); outer_left, k_left: how many there are.
  __device__ __forceinline__ void load(const E* p, int64_t ld, int64_t k0, int64_t k_left,
                                       int64_t outer_left, int tid) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = tid + i * THREADS;
      const int row = c / kPer;
      const int e = c % kPer * V;
      if constexpr (L == kRows) {
        const int64_t n = row < outer_left ? k_left - e : 0;
        r[i].load(p + row * ld + (k0 + e), n < V ? static_cast<int>(n) : V);
      } else {
        const int64_t n = row < k_left ? outer_left - e : 0;
        r[i].load(p + (k0 + row) * ld + e, n < V ? static_cast<int>(n) : V);
      }
    }
  }
  __device__ __forceinline__ void store(unsigned char* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = tid + i * THREADS;
      *reinterpret_cast<uint4*>(lds + slot(c / kPer, c % kPer)) = __builtin_bit_cast(uint4, r[i].q);
    }
  }
};

// Eight consecutive k of one row or column (bf16: k = 16 kk + 8 (lane / 32)).
template <typename S, Layout L>
__device__ __forceinline__ bf16x8_t frag_bf16(const unsigned char* lds, int outer, int kk, int lane) {
  if constexpr (L == kRows) {
    return *reinterpret_cast<const bf16x8_t*>(lds + S::slot(outer + (lane & 31), kk * 2 + (lane >> 5)));
  } else {
    typedef short v4i16_t __attribute__((ext_vector_type(4)));
    typedef short v8i16_t __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) v4i16_t* lds_v4_t;
    // ds_read_b64_tr_b16 as KMajorBOp uses it
    const int row = kk * 16 + ((lane >> 5) << 3) + ((lane >> 2) & 3);
    const int col = outer + (lane & 16) + ((lane & 3) << 2);
    const unsigned char* at = lds + S::slot(row, col >> 3) + ((col & 7) << 1);
    const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4_t)at);
    const v4i16_t hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4_t)(at + 4 * S::kPitch * 2));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// Four k of one row or column (float32: k = 8 q + 4 (lane / 32) + 0..3; which
// k a lane half has does not matter as long as A and B agree).
template <typename S, Layout L>
__device__ __forceinline__ void frag_f32(float (&f)[4], const unsigned char* lds, int outer, int q,
                                         int lane) {
  const float* p = reinterpret_cast<const float*>(lds);
  const int o = outer + (lane & 31), k = q * 8 + (lane >> 5) * 4;
  if constexpr (L == kRows) {
    const float4 v = *reinterpret_cast<const float4*>(p + o * S::kPitch + k);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = p[(k + i) * S::kPitch + o];
  }
}

template <typename E, int BM_, int BN_, int WM_, int WN_>
struct AnyCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = sizeof(E) == 2 ? 32 : 16;
  static constexpr int kWavesM = BM / WM, kWavesN = BN / WN;
  static constexpr int kThreads = kWavesM * kWavesN * kWave;
  static constexpr int kTm = WM / 32, kTn = WN / 32;
};

template <typename E, ProductKind KIND, bool PAIR, class C>
struct AnyParts {
  static constexpr Layout kA = KIND == kProductTN ? kKMajor : kRows;
  static constexpr Layout kB = KIND == kProductNT ? kRows : kKMajor;
  static constexpr int kBlocks = PAIR ? 2 : 1;
  using SA = Stager<E, C::BM, C::BK, kA, C::kThreads>;
  using SB = Stager<E, C::BN / kBlocks, C::BK, kB, C::kThreads>;
  static constexpr int kStage = SA::kBytes + kBlocks * SB::kBytes;
  static constexpr size_t kLds = 2 * kStage > band_bytes<C>() ? 2 * kStage : band_bytes<C>();
};

// `steps` K steps of BK to a slice (all of them without slices); with
// kPairSum the second segment's steps follow the first's.
template <typename E, ProductKind KIND, ProductPair PAIR, class C, class Epi>
__global__ __launch_bounds__(C::kThreads) void product_any_kernel(Product p, Epi epi, int tiles_m,
                                                                  int tiles_n, int steps) {
  constexpr bool kTwo = PAIR == kPairColumns;
  using P = AnyParts<E, KIND, kTwo, C>;
  extern __shared__ __align__(16) unsigned char lds[];
  // (the product on planes has been made)
  if (p.bad.word && *p.bad.word != p.bad.call) return;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = tid / kWave;
  const int wm = wave / C::kWavesN;
  const int wn = wave % C::kWavesN;
  const TileAt at = tile_at(tiles_m, tiles_n, PAIR == kPairTwo ? 2 : 1);
  constexpr int kCols = C::BN / P::kBlocks;
  const int64_t m0 = int64_t(at.tm) * C::BM;
  const int n0 = at.tn * kCols;
  const int64_t m_left = p.M - m0, n_left = p.N - n0;
  const E* a = static_cast<const E*>(p.a) + (P::kA == kRows ? m0 * p.lda : m0);
  const int64_t b0 = P::kB == kRows ? int64_t(n0) * p.ldb : n0;
  typename P::SA sa;
  typename P::SB sb[P::kBlocks];
  const int per = static_cast<int>((p.K + C::BK - 1) / C::BK);  // steps of one segment
  const int total = PAIR == kPairSum ? 2 * per : per;
  const int first = at.slice * steps;
  const int last = first + steps < total ? first + steps : total;
  auto load = [&](int ks) {
    const int seg = PAIR == kPairSum && ks >= per ? 1 : 0;
    const int64_t k0 = int64_t(ks - seg * per) * C::BK;
    sa.load(a + seg * p.a_second, p.lda, k0, p.K - k0, m_left, tid);
#pragma unroll
    for (int h = 0; h < P::kBlocks; ++h) {
      const void* b = p.b[PAIR == kPairSum ? seg : PAIR == kPairTwo ? at.which : h];
      sb[h].load(static_cast<const E*>(b) + b0, p.ldb, k0, p.K - k0, n_left, tid);
    }
  };
  auto store = [&](unsigned char* stage) {
    sa.store(stage, tid);
#pragma unroll
    for (int h = 0; h < P::kBlocks; ++h) sb[h].store(stage + P::SA::kBytes + h * P::SB::kBytes, tid);
  };
  f32x16_t acc[C::kTm][C::kTn];
#pragma unroll
  for (int i = 0; i < C::kTm; ++i)
#pragma unroll
    for (int j = 0; j < C::kTn; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  if (first < last) {
    load(first);
    store(lds);
    __syncthreads();
  }
  for (int ks = first; ks < last; ++ks) {
    const int cur = (ks - first) & 1;
    if (ks + 1 < last) load(ks + 1);
    const unsigned char* As = lds + cur * P::kStage;
    const unsigned char* Bs = As + P::SA::kBytes;
    // A gated pair's column block j is of operand j.
    auto b_at = [&](int j) { return Bs + (kTwo ? j * P::SB::kBytes : 0); };
    auto b_col = [&](int j) { return kTwo ? wn * 32 : wn * C::WN + j * 32; };
    if constexpr (sizeof(E) == 2) {
#pragma unroll
      for (int kk = 0; kk < C::BK / 16; ++kk) {
        bf16x8_t fa[C::kTm], fb[C::kTn];
#pragma unroll
        for (int i = 0; i < C::kTm; ++i)
          fa[i] = frag_bf16<typename P::SA, P::kA>(As, wm * C::WM + i * 32, kk, lane);
#pragma unroll
        for (int j = 0; j < C::kTn; ++j)
          fb[j] = frag_bf16<typename P::SB, P::kB>(b_at(j), b_col(j), kk, lane);
#pragma unroll
        for (int i = 0; i < C::kTm; ++i)
#pragma unroll
          for (int j = 0; j < C::kTn; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int q = 0; q < C::BK / 8; ++q) {
        float fa[C::kTm][4], fb[C::kTn][4];
#pragma unroll
        for (int i = 0; i < C::kTm; ++i)
          frag_f32<typename P::SA, P::kA>(fa[i], As, wm * C::WM + i * 32, q, lane);
#pragma unroll
        for (int j = 0; j < C::kTn; ++j)
          frag_f32<typename P::SB, P::kB>(fb[j], b_at(j), b_col(j), q, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < C::kTm; ++i)
#pragma unroll
            for (int j = 0; j < C::kTn; ++j)
              acc[i][j] =
                  __builtin_amdgcn_mfma_f32_32x32x2f32(fb[j][e], fa[i][e], acc[i][j], 0, 0, 0);
      }
    }
    if (ks + 1 < last) store(lds + (cur ^ 1) * P::kStage);
    __syncthreads();
  }
  if constexpr (std::is_same<Epi, PartialEpilogue<Epi::kGated>>::value) epi.slice(at.slice);
  tile_epilogue<C>(acc, lds, epi, m0, p.M, n0, p.N, at.which);
}

}  // namespace fff
