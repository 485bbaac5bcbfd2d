// How a product is cut and launched; one translation unit for each kind.
#pragma once

#include <type_traits>

#include "dense.hpp"
#include "dense_any.hpp"
#include "dense_direct.hpp"
#include "launch.hpp"

namespace fff {

// Kernels: register staged (any sizes, types and alignment) with tiles of 128 x
// 256 or, float32, 64 x 128, or straight into LDS with tiles of 256 x 256, 128
// x 256 or 128 x 128.
enum ProductTile { kTileAny, kTileAnySmall, kTileBig, kTileMid, kTileSmall };

struct Cut {
  ProductTile tile;
  int64_t tiles_m, tiles_n;
  int products;       // sums of a slice in the workspace
  int slices, steps;  // of K
};
Cut cut_product(const Product& p);
// In tiles of any sizes, K in one piece.
Cut cut_whole(const Product& p);

template <typename E> using TileAny = AnyCfg<E, 128, 256, 64, 64>;
using TileAnySmall = AnyCfg<float, 64, 128, 32, 64>;
using TileBig = StepCfg<256, 256, 128, 64, 3>;
using TileMid = StepCfg<128, 256, 64, 64, 4>;
using TileSmall = StepCfg<128, 128, 64, 64, 3>;  // two workgroups a compute unit

// The slices' sums through the epilogue (nothing where `bad` holds the call's number).
template <class Epi>
hipError_t launch_sum_slices(const float* partial, const Cut& c, int64_t M, int N, const Epi& epi,
                             const BeyondPlanes& bad, hipStream_t st);

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class Kernel, class Epi>
hipError_t launch_tiles(Kernel kern, size_t lds, int threads, const Product& p, const Epi& epi,
                        const Cut& c, hipStream_t st) {
  const hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), static_cast<int>(lds));
  if (e != hipSuccess) return e;
  const int64_t blocks = c.tiles_m * c.tiles_n * c.slices * (p.pair == kPairTwo ? 2 : 1);
  kern<<<dim3(static_cast<uint32_t>(blocks)), dim3(threads), lds, st>>>(
      p, epi, static_cast<int>(c.tiles_m), static_cast<int>(c.tiles_n), c.steps);
  return hipGetLastError();
}

// In tiles straight into LDS: bf16 operands, or (SIX) float32 ones' planes.
template <bool SIX, ProductKind KIND, ProductPair PAIR, class Epi>
hipError_t launch_direct(const Product& p, const Epi& epi, const Cut& c, hipStream_t st) {
  constexpr bool kTwo = PAIR == kPairColumns;
  auto direct = [&](auto cfg) {
    using C = decltype(cfg);
    return launch_tiles(product_direct_kernel<SIX, KIND, PAIR, C, Epi>,
                        DirectParts<KIND, kTwo, C>::kLds, C::kThreads, p, epi, c, st);
  };
  if (c.tile == kTileBig) return direct(TileBig());
  if constexpr (!kTwo) {
    if (c.tile == kTileSmall) return direct(TileSmall());
  }
  return direct(TileMid());
}

template <typename E, ProductKind KIND, ProductPair PAIR, class Epi>
hipError_t launch_cut(const Product& p, const Epi& epi, const Cut& c, hipStream_t st) {
  constexpr bool kTwo = PAIR == kPairColumns;
  auto any = [&](auto cfg) {
    using C = decltype(cfg);
    return launch_tiles(product_any_kernel<E, KIND, PAIR, C, Epi>, AnyParts<E, KIND, kTwo, C>::kLds,
                        C::kThreads, p, epi, c, st);
  };
  if (c.tile == kTileAny) return any(TileAny<E>());
  if constexpr (sizeof(E) == 4 && !kTwo) {
    if (c.tile == kTileAnySmall) return any(TileAnySmall());
  }
  return launch_direct<sizeof(E) == 4, KIND, PAIR>(p, epi, c, st);
}

template <typename E, ProductKind KIND, ProductPair PAIR, class Epi>
hipError_t run_with(const Product& p, const Epi& epi, void* workspace, hipStream_t st) {
  const Cut c = cut_product(p);
  hipError_t e;
  if (c.slices <= 1) {
    e = launch_cut<E, KIND, PAIR>(p, epi, c, st);
  } else {
    PartialEpilogue<Epi::kGated> part;
    part.partial = static_cast<float*>(workspace);
    part.M = p.M;
    part.N = p.N;
    part.products = c.products;
    e = launch_cut<E, KIND, PAIR>(p, part, c, st);
    if (e == hipSuccess) e = launch_sum_slices(part.partial, c, p.M, p.N, epi, p.bad, st);
  }
  // On planes: the kernel on the values themselves, should one be beyond them.
  if (e == hipSuccess && p.bad.word)
    e = launch_cut<E, KIND, PAIR>(p, epi, cut_whole(p), st);
  return e;
}

// Out and residual in the layer's type or in 32 bits.
template <typename E, ProductKind KIND, ProductPair PAIR>
hipError_t run_linear(const Product& p, void* workspace, hipStream_t st) {
  if constexpr (sizeof(E) == 2) {
    if (p.out_bf16) return run_with<E, KIND, PAIR>(p, LinearEpilogue<E, uint16_t>{p.e}, workspace, st);
  }
  return run_with<E, KIND, PAIR>(p, LinearEpilogue<E, float>{p.e}, workspace, st);
}

// Few rows (dense_small.hpp).
bool small_product(const Product& p);
size_t small_workspace(const Product& p);
hipError_t launch_small(const Product& p, void* workspace, hipStream_t st);

hipError_t run_nn(const Product& p, void* workspace, hipStream_t st);
hipError_t run_nt(const Product& p, void* workspace, hipStream_t st);
hipError_t run_tn(const Product& p, void* workspace, hipStream_t st);

}  // namespace fff
