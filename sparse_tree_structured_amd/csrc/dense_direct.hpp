// bf16 product whose operands go straight from memory into LDS.
//
// Needs 16-byte aligned operands and rows of whole 16-byte pieces.  The
// stages, their swizzles and the schedule are those of
// gemm_mainloop_direct_op (mfma_tile.hpp); here either operand is K contiguous
// or k-major, two B operands can lie side by side or follow one another along
// K, and K ends anywhere: in the last step the pieces past it come from 16
// zero bytes.  A copy takes a uniform base and 32 bits of offset for each
// lane, which stay the same over the loop.
#pragma once

#include "dense.hpp"
#include "dense_any.hpp"

namespace fff {

static __device__ __align__(16) const unsigned char kZeros[16] = {};

// dma16_asm with the address as a uniform base and a lane's offset.
__device__ __forceinline__ void dma16_base(const void* base, uint32_t offset, uint32_t lds_at) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(offset), "s"(base), "s"(lds_at)
      : "memory");
}

// Where a lane's 16 bytes of 1 KB piece q of a stage's block of OUTER rows
// (or columns) by 32 of K come from: rows (or columns) outer, K from k on.
template <int OUTER, Layout L>
struct PieceAt {
  int outer, k;
  __device__ __forceinline__ PieceAt(int q, int lane) {
    if constexpr (L == kRows) {
      outer = q * 16 + (lane >> 2);
      k = ((lane & 3) ^ lds_swz(outer)) * 8;
    } else {
      constexpr int kRow = OUTER * 2;
      const int byte = q * 1024 + lane * 16;
      k = byte / kRow;
      outer = (((byte % kRow) >> 4) ^ ((k & 3) << 2)) * 8;
    }
  }
  // Bytes from the block's first element; what is past the operand's end is
  // read from its last row, or its first columns, and not used.
  __device__ __forceinline__ uint32_t offset(int64_t ld, int64_t left) const {
    if constexpr (L == kRows) {
      const int r = outer < left ? outer : static_cast<int>(left) - 1;
      return (static_cast<uint32_t>(r) * static_cast<uint32_t>(ld) + k) * 2;
    } else {
      return (static_cast<uint32_t>(k) * static_cast<uint32_t>(ld) + (outer < left ? outer : 0)) * 2;
    }
  }
};

template <ProductKind KIND, bool PAIR, class C>
struct DirectParts {
  static constexpr Layout kA = KIND == kProductTN ? kKMajor : kRows;
  static constexpr Layout kB = KIND == kProductNT ? kRows : kKMajor;
  static constexpr int kBlocks = PAIR ? 2 : 1;
  static constexpr int kBCols = C::BN / kBlocks;
  static constexpr int kBPieces = kBCols / 16;  // of one block
  using SA = Stager<uint16_t, C::BM, 32, kA, C::BM * 4>;
  using SB = Stager<uint16_t, kBCols, 32, kB, kBCols * 4>;
  static constexpr size_t kLds = C::kLdsBytes > band_bytes<C>() ? C::kLdsBytes : band_bytes<C>();
  static_assert(SA::kBytes == C::BM * 64 && SB::kBytes == kBCols * 64, "stage blocks");
};

template <ProductKind KIND, ProductPair PAIR, class C, class Epi>
__global__ __launch_bounds__(C::kThreads) void product_direct_kernel(Product p, Epi epi, int tiles_m,
                                                                     int tiles_n, int steps) {
  constexpr bool kTwo = PAIR == kPairColumns;
  using P = DirectParts<KIND, kTwo, C>;
  constexpr int S = C::kStages;
  constexpr int kPerStage = C::kALoads + C::kBLoads;
  extern __shared__ __align__(16) unsigned char lds[];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / C::kWavesN;
  const int wn = wave % C::kWavesN;
  const TileAt at = tile_at(tiles_m, tiles_n, PAIR == kPairTwo ? 2 : 1);
  const int64_t m0 = int64_t(at.tm) * C::BM;
  const int n0 = at.tn * P::kBCols;
  const uint32_t lds_at = __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)));
  uint32_t a_off[C::kALoads], b_off[C::kBLoads];
#pragma unroll
  for (int j = 0; j < C::kALoads; ++j)
    a_off[j] = PieceAt<C::BM, P::kA>(wave * C::kALoads + j, lane).offset(p.lda, p.M - m0);
#pragma unroll
  for (int j = 0; j < C::kBLoads; ++j)
    b_off[j] = PieceAt<P::kBCols, P::kB>((wave * C::kBLoads + j) % P::kBPieces, lane)
                   .offset(p.ldb, p.N - n0);
  const int64_t a_step = P::kA == kRows ? 64 : p.lda * 64;  // bytes from a step to the next
  const int64_t b_step = P::kB == kRows ? 64 : p.ldb * 64;
  const unsigned char* a0 =
      static_cast<const unsigned char*>(p.a) + 2 * (P::kA == kRows ? m0 * p.lda : m0);
  const int64_t b0 = 2 * (P::kB == kRows ? int64_t(n0) * p.ldb : n0);
  const int per = static_cast<int>((p.K + 31) / 32);  // steps of one segment
  const int total = PAIR == kPairSum ? 2 * per : per;
  const int first = at.slice * steps;
  const int nk = (first + steps < total ? first + steps : total) - first;

  auto issue = [&](int s) {
    const int ks = first + s;
    const int seg = PAIR == kPairSum && ks >= per ? 1 : 0;
    const int k = ks - seg * per;
    const unsigned char* a = a0 + k * a_step + (PAIR == kPairSum ? seg * p.a_second * 2 : 0);
    const int64_t k_left = p.K - int64_t(k) * 32;
    const uint32_t stage = lds_at + (s % S) * C::kStageBytes;
    auto copy = [&](const void* base, uint32_t offset, uint32_t to, bool there) {
      if (k_left >= 32) {
        dma16_base(base, offset, to);
      } else {
        const unsigned char* from = static_cast<const unsigned char*>(base) + offset;
        if (!there) from = kZeros;
        dma16_asm(from, reinterpret_cast<unsigned char*>(static_cast<uintptr_t>(to)));
      }
    };
#pragma unroll
    for (int j = 0; j < C::kALoads; ++j) {
      const int q = wave * C::kALoads + j;
      copy(a, a_off[j], stage + q * 1024, PieceAt<C::BM, P::kA>(q, lane).k < k_left);
    }
#pragma unroll
    for (int j = 0; j < C::kBLoads; ++j) {
      const int q = wave * C::kBLoads + j;
      const int which = PAIR == kPairSum ? seg : PAIR == kPairTwo ? at.which : q / P::kBPieces;
      const unsigned char* b =
          static_cast<const unsigned char*>(which ? p.b[1] : p.b[0]) + b0 + k * b_step;
      copy(b, b_off[j], stage + C::BM * 64 + q * 1024,
           PieceAt<P::kBCols, P::kB>(q % P::kBPieces, lane).k < k_left);
    }
  };
  auto read = [&](Frags<C>& f, int s, int kk) {
    const unsigned char* As = lds + (s % S) * C::kStageBytes;
    const unsigned char* Bs = As + C::BM * 64;
#pragma unroll
    for (int i = 0; i < C::kTm; ++i)
      f.a[i] = frag_bf16<typename P::SA, P::kA>(As, wm * C::WM + i * 32, kk, lane);
#pragma unroll
    for (int j = 0; j < C::kTn; ++j)
      f.b[j] = frag_bf16<typename P::SB, P::kB>(Bs + (kTwo ? j * P::SB::kBytes : 0),
                                               kTwo ? wn * 32 : wn * C::WN + j * 32, kk, lane);
  };

  f32x16_t acc[C::kTm][C::kTn];
  zero_acc<C>(acc);
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < nk) issue(s);
  wait_stages<kPerStage, S - 2>(nk - 1);
  stage_barrier();
  Frags<C> f0, f1;
  read(f0, 0, 0);
  for (int s = 0; s < nk; ++s) {
    read(f1, s, 1);
    asm volatile("" ::: "memory");
    mma_frags<C>(acc, f0);
    if (s + 1 < nk) {
      wait_stages<kPerStage, S - 3>(nk - 2 - s);
      stage_barrier();
      if (s + S - 1 < nk) issue(s + S - 1);
    }
    read(f0, s + 1, 0);
    asm volatile("" ::: "memory");
    mma_frags<C>(acc, f1);
  }
  __syncthreads();
  if constexpr (std::is_same<Epi, PartialEpilogue<Epi::kGated>>::value) epi.slice(at.slice);
  tile_epilogue<C>(acc, lds, epi, m0, p.M, n0, p.N, at.which);
}

}  // namespace fff
