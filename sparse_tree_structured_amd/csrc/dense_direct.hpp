// bf16 product whose operands go straight from memory into LDS.
//
// Needs 16-byte aligned operands and rows of whole 16-byte pieces.  Either
// operand is K contiguous or k-major, two B operands can lie side by side or
// follow one another along K, and K ends anywhere: in the last step the
// pieces past it come from 16 zero bytes.
//
// A step is 64 of K (a K-contiguous row's piece is a whole 128-byte line).
// Once a stage's last fragments are in registers, its buffers take the stages
// as far ahead as there are buffers.  Copies and fragment reads are issued one
// by one between matrix-core operations, and a copy is one instruction with a
// uniform base, made once a stage, and 32 bits of offset for each lane that
// stay the same over the loop: with the copies in one piece and their
// addresses made for each, the matrix cores had work in 57 % of the cycles.
//
// Bound by the matrix cores and the power they take: over K = 16384 they have
// work in 77 % of the cycles (da . W^T), 75 % (x^T . da), and over K = 2048 in
// 64 % (x . W, 16384 columns), at a clock that the load brings down to 1.55 to
// 1.65 GHz of 2.4.  16384 x 8192 x 8192: x . W 1.25 to 1.31 PFLOP/s by board,
// da . W^T 1.24, x^T . da 1.29 to 1.35.  Tried and left out: four wavefronts of 128
// x 128 (7 % slower), 16 x 16 x 32 operations (the same), steps of 32 in four
// or five stages (4 %), all copies in a stage's last phase (2 %).
#pragma once

#include "dense.hpp"
#include "dense_any.hpp"
#include "dense_epilogue.hpp"

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

// Tiles of BM x BN, a wavefront WM x WN of them, with A_STAGES buffers of A and
// one fewer of B.
template <int BM_, int BN_, int WM_, int WN_, int A_STAGES>
struct StepCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 64;
  static constexpr int kAStages = A_STAGES, kBStages = A_STAGES - 1;
  static_assert(kBStages >= 2, "a stage is filled while another is used");
  static constexpr int kWavesM = BM / WM, kWavesN = BN / WN, kWaves = kWavesM * kWavesN;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kTm = WM / 32, kTn = WN / 32;
  static constexpr int kABytes = BM * BK * 2, kBBytes = BN * BK * 2;  // of a stage
  static constexpr size_t kLdsBytes = size_t(kAStages) * kABytes + size_t(kBStages) * kBBytes;
  static constexpr int kALoads = BM * BK / 512 / kWaves;  // 1 KB copies of a wavefront and stage
  static constexpr int kBLoads = BN * BK / 512 / kWaves;
  static_assert(BM * BK % (512 * kWaves) == 0 && BN * BK % (512 * kWaves) == 0, "whole copies");
};

// f(0), f(1), ... f(N - 1) with constants.
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(const F& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    each<N, I + 1>(f);
  }
}

// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const unsigned char* uniform(const unsigned char* p) {
  const uintptr_t v = reinterpret_cast<uintptr_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const unsigned char*>(static_cast<uintptr_t>(hi) << 32 | lo);
}

// Where a lane's 16 bytes of 1 KB piece q of a stage's block of OUTER rows
// (or columns) by BK of K come from: rows (or columns) outer, K from k on.
template <int OUTER, int BK, Layout L>
struct PieceAt {
  int outer, k;
  __device__ __forceinline__ PieceAt(int q, int lane) {
    using S = Stager<uint16_t, OUTER, BK, L, OUTER * BK / 8>;
    constexpr int kRow = L == kRows ? BK * 2 : OUTER * 2;
    const int byte = q * 1024 + lane * 16;
    const int row = byte / kRow;
    const int e = (((byte % kRow) >> 4) ^ S::swizzle(row)) * 8;
    outer = L == kRows ? row : e;
    k = L == kRows ? e : row;
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
  static constexpr int kBPieces = kBCols * C::BK / 512;  // of one block
  using SA = Stager<uint16_t, C::BM, C::BK, kA, C::BM * C::BK / 8>;
  using SB = Stager<uint16_t, kBCols, C::BK, kB, kBCols * C::BK / 8>;
  using PA = PieceAt<C::BM, C::BK, kA>;
  using PB = PieceAt<kBCols, C::BK, kB>;
  static constexpr size_t most(size_t a, size_t b) { return a > b ? a : b; }
  static constexpr size_t out_bytes() {
    if constexpr (PAIR) return most(GatedStage<C>::kBytes, band_bytes<C>());
    return most(LinearStage<C>::kBytes, band_bytes<C>());
  }
  static constexpr size_t kLds = most(C::kLdsBytes, out_bytes());
  static_assert(kLds <= 160 * 1024, "LDS of a workgroup");
  static_assert(SA::kBytes == C::BM * C::BK * 2 && SB::kBytes == kBCols * C::BK * 2, "stage blocks");
};

// SIX: the operands are the planes of float32 ones, h + m + l each, and K is
// gone through six times: l h + h l + m m + m h + h m + h h, the small terms
// first.  What is left out is about 2^-24 of the sizes' product, as one
// rounding of a 32-bit product is; the matrix cores' bf16 rate is 16 times
// their float32 rate, so this is worth 6 / 16 of it and the planes.
constexpr uint32_t kSixA = 0x052;  // two bits a term: 2 0 1 1 0 0
constexpr uint32_t kSixB = 0x118;  //                  0 2 1 0 1 0

template <bool SIX, ProductKind KIND, ProductPair PAIR, class C, class Epi>
__global__ __launch_bounds__(C::kThreads) void product_direct_kernel(Product p, Epi epi, int tiles_m,
                                                                     int tiles_n, int steps) {
  constexpr bool kTwo = PAIR == kPairColumns;
  using P = DirectParts<KIND, kTwo, C>;
  constexpr int kACopies = C::kALoads, kBCopies = C::kBLoads;
  constexpr int kTerms = SIX ? 6 : 1;
  extern __shared__ __align__(16) unsigned char lds[];
  if (SIX && *p.bad.word == p.bad.call) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / C::kWavesN;
  const int wn = wave % C::kWavesN;
  const TileAt at = tile_at(tiles_m, tiles_n, PAIR == kPairTwo ? 2 : 1);
  const int64_t m0 = int64_t(at.tm) * C::BM;
  const int n0 = at.tn * P::kBCols;
  const int64_t lda = SIX ? p.a_planes.ld : p.lda;
  const int64_t ldb = SIX ? p.b_planes[0].ld : p.ldb;
  const int64_t a_second = SIX ? p.a_planes_second : p.a_second;
  const void* const b_first = SIX ? p.b_planes[0].at : p.b[0];
  const void* const b_other = SIX ? p.b_planes[1].at : p.b[1];
  const uint32_t lds_at = __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)));
  uint32_t a_off[C::kALoads], b_off[C::kBLoads];
#pragma unroll
  for (int j = 0; j < C::kALoads; ++j)
    a_off[j] = typename P::PA(wave * C::kALoads + j, lane).offset(lda, p.M - m0);
#pragma unroll
  for (int j = 0; j < C::kBLoads; ++j)
    b_off[j] = typename P::PB((wave * C::kBLoads + j) % P::kBPieces, lane).offset(ldb, p.N - n0);
  const int64_t a_step = P::kA == kRows ? C::BK * 2 : lda * (C::BK * 2);  // bytes from a step to the next
  const int64_t b_step = P::kB == kRows ? C::BK * 2 : ldb * (C::BK * 2);
  const unsigned char* a0 =
      static_cast<const unsigned char*>(SIX ? p.a_planes.at : p.a) +
      2 * (P::kA == kRows ? m0 * lda : m0);
  const int64_t b0 = 2 * (P::kB == kRows ? int64_t(n0) * ldb : n0);
  const int per = static_cast<int>((p.K + C::BK - 1) / C::BK);  // steps of one segment of K
  const int total = per * kTerms * (PAIR == kPairSum ? 2 : 1);
  const int first = at.slice * steps;
  const int nk = (first + steps < total ? first + steps : total) - first;

  // Where the copies of an operand's next stage come from and go to, the same
  // for all lanes: asked for once for every stage, in their order.
  struct From {
    const unsigned char *p0, *p1;
    uint32_t to;
    int k_left;
  };
  struct Next {
    int seg, k;  // segment of K and step in it
  };
  const int seg0 = kTerms == 1 && PAIR != kPairSum ? 0 : first / (per > 0 ? per : 1);
  Next next_a = {seg0, first - seg0 * per}, next_b = next_a;
  auto step = [&](Next& n) __attribute__((always_inline)) {
    if (++n.k == per) {
      n.k = 0;
      ++n.seg;
    }
  };
  auto term_of = [&](const Next& n) __attribute__((always_inline)) {
    return PAIR == kPairSum && n.seg >= kTerms ? n.seg - kTerms : n.seg;
  };
  auto from_a = [&](int s) __attribute__((always_inline)) {
    int64_t at = next_a.k * a_step;
    if constexpr (SIX) at += (kSixA >> (2 * term_of(next_a)) & 3) * p.a_planes.plane * 2;
    if (PAIR == kPairSum && next_a.seg >= kTerms) at += a_second * 2;
    From f;
    f.p0 = uniform(a0 + at);
    f.p1 = nullptr;
    f.to = __builtin_amdgcn_readfirstlane(lds_at + (s % C::kAStages) * C::kABytes);
    f.k_left = static_cast<int>(p.K) - next_a.k * C::BK;
    step(next_a);
    return f;
  };
  auto from_b = [&](int s) __attribute__((always_inline)) {
    int64_t at_b = b0 + next_b.k * b_step;
    if constexpr (SIX) at_b += (kSixB >> (2 * term_of(next_b)) & 3) * p.b_planes[0].plane * 2;
    const bool second = PAIR == kPairSum ? next_b.seg >= kTerms : PAIR == kPairTwo && at.which != 0;
    From f;
    f.p0 = uniform(static_cast<const unsigned char*>(second ? b_other : b_first) + at_b);
    f.p1 = kTwo ? uniform(static_cast<const unsigned char*>(b_other) + at_b) : nullptr;
    f.to = __builtin_amdgcn_readfirstlane(lds_at + C::kAStages * C::kABytes +
                                          (s % C::kBStages) * C::kBBytes);
    f.k_left = static_cast<int>(p.K) - next_b.k * C::BK;
    step(next_b);
    return f;
  };
  // Copy j of a wavefront; TAIL: the operand may end in the stage.
  auto copy = [&](const From& f, const unsigned char* base, uint32_t offset, uint32_t to, int piece_k,
                  auto tail) __attribute__((always_inline)) {
    if constexpr (!decltype(tail)::value) {
      dma16_base(base, offset, to);
    } else {
      const unsigned char* at = piece_k < f.k_left ? base + offset : kZeros;
      dma16_asm(at, reinterpret_cast<unsigned char*>(static_cast<uintptr_t>(to)));
    }
  };
  auto copy_a = [&](const From& f, auto j, auto tail) __attribute__((always_inline)) {
    const int q = wave * kACopies + j;
    copy(f, f.p0, a_off[j], f.to + q * 1024, typename P::PA(q, lane).k, tail);
  };
  auto copy_b = [&](const From& f, auto j, auto tail) __attribute__((always_inline)) {
    const int q = wave * kBCopies + j;
    copy(f, kTwo && q >= P::kBPieces ? f.p1 : f.p0, b_off[j], f.to + q * 1024,
         typename P::PB(q % P::kBPieces, lane).k, tail);
  };
  auto fill_a = [&](int s) __attribute__((always_inline)) {
    if (s >= nk) return;
    const From f = from_a(s);
    each<kACopies>([&](auto j) __attribute__((always_inline)) { copy_a(f, j, std::true_type()); });
  };
  auto fill_b = [&](int s) __attribute__((always_inline)) {
    if (s >= nk) return;
    const From f = from_b(s);
    each<kBCopies>([&](auto j) __attribute__((always_inline)) { copy_b(f, j, std::true_type()); });
  };
  // Fragment n (of kFrags) of step kk of stage s, in the order of their first use.
  constexpr int kFrags = C::kTm + C::kTn;
  auto read = [&](Frags<C>& f, int s, int kk, auto frag_n) __attribute__((always_inline)) {
    constexpr int n = decltype(frag_n)::value;
    const unsigned char* As = lds + (s % C::kAStages) * C::kABytes;
    const unsigned char* Bs = lds + C::kAStages * C::kABytes + (s % C::kBStages) * C::kBBytes;
    if constexpr (n < C::kTn) {
      f.b[n] = frag_bf16<typename P::SB, P::kB>(
          Bs + (kTwo ? n / (C::kTn / 2) * P::SB::kBytes : 0),
          kTwo ? wn * (C::WN / 2) + n % (C::kTn / 2) * 32 : wn * C::WN + n * 32, kk, lane);
    } else {
      const int i = n - C::kTn;
      f.a[i] = frag_bf16<typename P::SA, P::kA>(As, wm * C::WM + i * 32, kk, lane);
    }
  };

  f32x16_t acc[C::kTm][C::kTn];
  zero_acc<C>(acc);
  Frags<C> f0, f1;
  // The matrix-core operations of one step of 16, with the fragments of the
  // next step read between them, and copies between those: bunched up, either
  // leaves the matrix cores without work while it is issued.
  constexpr int kMma = C::kTm * C::kTn;
  // (reads at the front: the last are back when a barrier follows)
  constexpr int kReadMma = kFrags < kMma ? kFrags : kMma;
  // Copies come in rounds: round s fills B of stage s + kBStages, then A of
  // stage s + kAStages, from the last phase of stage s to the third of the
  // next, evenly: the address unit has 27 cycles of work for each of the 64
  // copies that a compute unit makes in a stage of 2048 cycles.
  enum { kNoCopies, kWholeCopies, kAnyCopies };  // any: stages with a tail, or none
  using None = std::integral_constant<int, kNoCopies>;
  using Whole = std::integral_constant<int, kWholeCopies>;
  using Any = std::integral_constant<int, kAnyCopies>;
  constexpr int kCopies = kACopies + kBCopies;
  From fa, fb;
  bool has_a = false, has_b = false;
  auto start_round = [&](int s, auto copies) __attribute__((always_inline)) {
    if constexpr (decltype(copies)::value == kWholeCopies) {
      fb = from_b(s + C::kBStages);
      fa = from_a(s + C::kAStages);
    } else {
      has_b = s + C::kBStages < nk;
      has_a = s + C::kAStages < nk;
      if (has_b) fb = from_b(s + C::kBStages);
      if (has_a) fa = from_a(s + C::kAStages);
    }
  };
  // part: 0 to 3, the phase of the round.
  auto phase = [&](const Frags<C>& f, Frags<C>& next, int rs, int rkk, auto part, auto copies)
      __attribute__((always_inline)) {
    constexpr int kHow = decltype(copies)::value;
    each<kMma>([&](auto m) __attribute__((always_inline)) {
      constexpr int i = m / C::kTn, j = m % C::kTn;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
      each<kFrags>([&](auto n) __attribute__((always_inline)) {
        if constexpr (n * kReadMma / kFrags == m) read(next, rs, rkk, n);
      });
      each<kCopies>([&](auto c) __attribute__((always_inline)) {
        constexpr int kSlot = c * (4 * kMma - kMma / 2) / kCopies;
        if constexpr (kHow != kNoCopies && kSlot == decltype(part)::value * kMma + m) {
          using Tail = std::integral_constant<bool, kHow == kAnyCopies>;
          if constexpr (c < kBCopies) {
            if (kHow == kWholeCopies || has_b) copy_b(fb, c, Tail());
          } else {
            if (kHow == kWholeCopies || has_a)
              copy_a(fa, std::integral_constant<int, c - kBCopies>(), Tail());
          }
        }
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  using Part0 = std::integral_constant<int, 0>;
  using Part1 = std::integral_constant<int, 1>;
  using Part2 = std::integral_constant<int, 2>;
  using Part3 = std::integral_constant<int, 3>;
  auto read_all = [&](Frags<C>& f, int s, int kk) __attribute__((always_inline)) {
    each<kFrags>([&](auto n) __attribute__((always_inline)) { read(f, s, kk, n); });
  };
  // Before the last phase of stage s: its last fragments are in registers, and
  // stage s + 1 is there.  Behind its B are A's copies of the same round and
  // the rounds after it, up to s - 1.
  auto meet = [&](int s) __attribute__((always_inline)) {
    if (s + 1 >= nk) return;
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt 0
    if (s - 1 + C::kAStages < nk)
      wait_vmcnt<(C::kBStages - 2) * kCopies + kACopies>();
    else
      wait_vmcnt<0>();
    stage_barrier();
  };
  // The last phase of stage s - 1 and the first three of stage s.
  auto body = [&](int s, auto copies) __attribute__((always_inline)) {
    start_round(s - 1, copies);
    phase(f1, f0, s, 0, Part0(), copies);
    phase(f0, f1, s, 1, Part1(), copies);
    phase(f1, f0, s, 2, Part2(), copies);
    phase(f0, f1, s, 3, Part3(), copies);
    meet(s);
  };
  // The rounds before stage 0, without work.
#pragma unroll
  for (int s = -C::kAStages; s < 0; ++s) {
    if (s + C::kBStages >= 0) fill_b(s + C::kBStages);
    fill_a(s + C::kAStages);
  }
  if (nk > C::kAStages)
    wait_vmcnt<kCopies>();
  else
    wait_vmcnt<0>();
  stage_barrier();
  if (nk > 0) {
    read_all(f0, 0, 0);
    phase(f0, f1, 0, 1, Part1(), None());
    phase(f1, f0, 0, 2, Part2(), None());
    phase(f0, f1, 0, 3, Part3(), None());
    meet(0);
    // Runs of rounds that fill whole stages, and single ones that fill a tail or nothing.
    const bool tails = p.K % C::BK != 0;
    for (int s = 1; s < nk;) {
      int end = nk - C::kAStages + 1;  // round s - 1 fills A of stage s - 1 + kAStages
      if (tails) {
        const int whole = per - 1 - (next_a.k > next_b.k ? next_a.k : next_b.k);
        if (s + whole < end) end = s + whole;
      }
      for (; s < end; ++s) body(s, Whole());
      if (s < nk) body(s, Any());
      ++s;
    }
    mma_frags<C>(acc, f1);
  }
  __syncthreads();
  if constexpr (std::is_same<Epi, GatedEpilogue<uint16_t>>::value) {
    gated_epilogue<C>(acc, lds, epi.e, m0, n0);
  } else if constexpr (std::is_same<Epi, LinearEpilogue<uint16_t, uint16_t>>::value) {
    if (epi.e.save[0] ||
        (epi.e.residual && (p.N % 8 != 0 || reinterpret_cast<uintptr_t>(epi.e.residual) % 16 != 0)))
      tile_epilogue<C>(acc, lds, epi, m0, p.M, n0, p.N, at.which);
    else
      linear_epilogue<C>(acc, lds, epi.e, m0, n0, at.which);
  } else {
    if constexpr (std::is_same<Epi, PartialEpilogue<Epi::kGated>>::value) epi.slice(at.slice);
    tile_epilogue<C>(acc, lds, epi, m0, p.M, n0, p.N, at.which);
  }
}

}  // namespace fff
