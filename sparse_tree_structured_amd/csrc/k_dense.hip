// Matrix products of the dense feed-forward block: choice of kernel, slices
// of K and their sums.
#include <type_traits>

#include "dense.hpp"
#include "dense_any.hpp"
#include "launch.hpp"

namespace fff {
namespace {

// The slices' sums, added in their order, through the epilogue: a wavefront
// has 256 columns of a row.
template <class Epi>
__global__ __launch_bounds__(256) void sum_slices_kernel(const float* partial, int slices,
                                                         int products, int64_t M, int N, Epi epi) {
  const int lane = threadIdx.x & (kWave - 1);
  const int strips = (N + 255) / 256;
  const int64_t units = M * strips * (Epi::kGated ? 1 : products);
  for (int64_t u = int64_t(blockIdx.x) * 4 + threadIdx.x / kWave; u < units;
       u += int64_t(gridDim.x) * 4) {
    const int col = static_cast<int>(u % strips) * 256 + lane * 4;
    const int64_t row = u / strips % M;
    const int which = Epi::kGated ? 0 : static_cast<int>(u / strips / M);
    const int left = N - col;
    const int n = left < 0 ? 0 : left < 4 ? left : 4;
    typename Epi::Column column;
    typename Epi::Early early;
    epi.column(column, col);
    epi.early(early, row, col, n);
    float v[4] = {}, w[4] = {};
    for (int s = 0; s < slices; ++s) {
      const float* p = partial + ((static_cast<size_t>(s) * products + which) * M + row) * N + col;
      Pack<float, 4> q;
      q.load(p, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += q.get(i);
      if constexpr (Epi::kGated) {
        q.load(p + static_cast<size_t>(M) * N, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] += q.get(i);
      }
    }
    epi.apply(column, early, row, col, n, v, w, which);
  }
}

template <typename E> using TileAny = AnyCfg<E, 128, 256, 64, 64>;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a product is cut.
struct Cut {
  int64_t tiles_m, tiles_n;
  int products;  // sums of a slice in the workspace
  int slices, steps;
};

// Slices of K while the tiles leave compute units idle: as many as fill the
// chip once, of at least 8 steps each.
Cut cut_any(const Product& p) {
  const int bk = p.bf16 ? 32 : 16;
  Cut c;
  const int cols = p.pair == kPairColumns ? 128 : 256;
  c.tiles_m = ceil_div(p.M, 128);
  c.tiles_n = ceil_div(p.N, cols);
  c.products = p.pair == kPairColumns || p.pair == kPairTwo ? 2 : 1;
  int64_t tiles = c.tiles_m * c.tiles_n * (p.pair == kPairTwo ? 2 : 1);
  if (tiles < 1) tiles = 1;
  const int64_t total = ceil_div(p.K, bk) * (p.pair == kPairSum ? 2 : 1);
  int64_t slices = 1;
  if (tiles < 192) {
    slices = 256 / tiles;
    if (slices > total / 8) slices = total / 8;
    if (slices < 1) slices = 1;
  }
  c.steps = static_cast<int>(ceil_div(total, slices));
  c.slices = total > 0 ? static_cast<int>(ceil_div(total, c.steps)) : 1;
  return c;
}

template <typename E, ProductKind KIND, ProductPair PAIR, class Epi>
hipError_t run_any(const Product& p, const Epi& epi, const Cut& c, hipStream_t st) {
  using Cfg = TileAny<E>;
  auto kern = product_any_kernel<E, KIND, PAIR, Cfg, Epi>;
  constexpr size_t lds = AnyParts<E, KIND, PAIR == kPairColumns, Cfg>::kLds;
  const hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(kern), static_cast<int>(lds));
  if (e != hipSuccess) return e;
  const int64_t blocks = c.tiles_m * c.tiles_n * c.slices * (PAIR == kPairTwo ? 2 : 1);
  kern<<<dim3(static_cast<uint32_t>(blocks)), dim3(Cfg::kThreads), lds, st>>>(
      p, epi, static_cast<int>(c.tiles_m), static_cast<int>(c.tiles_n), c.steps);
  return hipGetLastError();
}

template <typename E, ProductKind KIND, ProductPair PAIR, class Epi>
hipError_t run_with(const Product& p, const Epi& epi, void* workspace, hipStream_t st) {
  const Cut c = cut_any(p);
  if (c.slices <= 1) return run_any<E, KIND, PAIR>(p, epi, c, st);
  PartialEpilogue<Epi::kGated> part;
  part.partial = static_cast<float*>(workspace);
  part.M = p.M;
  part.N = p.N;
  part.products = c.products;
  const hipError_t e = run_any<E, KIND, PAIR>(p, part, c, st);
  if (e != hipSuccess) return e;
  const int64_t units = p.M * ceil_div(p.N, 256) * (Epi::kGated ? 1 : c.products);
  const int64_t blocks = ceil_div(units, 4);
  sum_slices_kernel<Epi><<<dim3(static_cast<uint32_t>(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                           st>>>(part.partial, c.slices, c.products, p.M, p.N, epi);
  return hipGetLastError();
}

template <typename E, ProductKind KIND, ProductPair PAIR>
hipError_t run_linear(const Product& p, void* workspace, hipStream_t st) {
  if constexpr (sizeof(E) == 2) {
    if (p.out_bf16) return run_with<E, KIND, PAIR>(p, LinearEpilogue<E, uint16_t>{p.e}, workspace, st);
  }
  return run_with<E, KIND, PAIR>(p, LinearEpilogue<E, float>{p.e}, workspace, st);
}

template <typename E>
hipError_t run_product(const Product& p, void* workspace, hipStream_t st) {
  if (p.kind == kProductNN) {
    if (p.pair == kPairColumns)
      return run_with<E, kProductNN, kPairColumns>(p, GatedEpilogue<E>{p.e}, workspace, st);
    return run_linear<E, kProductNN, kSingle>(p, workspace, st);
  }
  if (p.kind == kProductNT) {
    if (p.pair == kPairSum) return run_linear<E, kProductNT, kPairSum>(p, workspace, st);
    return run_linear<E, kProductNT, kSingle>(p, workspace, st);
  }
  if (p.pair == kPairTwo) return run_linear<E, kProductTN, kPairTwo>(p, workspace, st);
  return run_linear<E, kProductTN, kSingle>(p, workspace, st);
}

}  // namespace

bool product_fits(const Product& p) {
  const Cut c = cut_any(p);
  // (a launch has fewer than 2^32 threads)
  return c.tiles_m * c.tiles_n * c.slices * 2 < (int64_t(1) << 23);
}

size_t product_workspace(const Product& p) {
  const Cut c = cut_any(p);
  return c.slices <= 1 ? 0
                       : size_t(c.slices) * c.products * size_t(p.M) * size_t(p.N) * sizeof(float);
}

hipError_t launch_product(const Product& p, void* workspace, hipStream_t st) {
  return p.bf16 ? run_product<uint16_t>(p, workspace, st) : run_product<float>(p, workspace, st);
}

}  // namespace fff
