// Products x . W of few rows: choice of slices, launches.
#include <atomic>
#include <chrono>

#include "dense_small.hpp"
#include "product.hpp"

namespace fff {
namespace {

int64_t col_blocks(const Product& p) { return ceil_div(p.N, kSmallCols); }

// Slices of K: as many as give every compute unit a workgroup, with at least
// a step for each wavefront.  Twice as many take longer to meet than their
// loads gain: 1 x 8192 x 2048 13.3 us instead of 11.6, 64 rows 28 instead of 20.
int slices_of(const Product& p) {
  const int64_t steps = ceil_div(p.K, kSmallStep);
  int64_t s = 256 / col_blocks(p);
  if (s > steps / kSmallWaves) s = steps / kSmallWaves;
  if (s > kSmallMaxSlices) s = kSmallMaxSlices;
  return s < 1 ? 1 : static_cast<int>(s);
}

// Floats that the arrivals' words take.
int64_t word_floats(int64_t blocks, int64_t slices) { return (blocks * (slices + 1) * 2 + 63) / 64 * 64; }

int row_tiles(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }

template <typename E, int TT, class Epi>
hipError_t launch(const Product& p, const Epi& epi, void* workspace, hipStream_t st) {
  const int64_t blocks = col_blocks(p);
  const int64_t total = ceil_div(p.K, kSmallStep);
  const int64_t steps = ceil_div(total, slices_of(p));
  const int slices = static_cast<int>(ceil_div(total, steps));
  auto kern = product_small_kernel<E, TT, Epi>;
  const hipError_t e =
      ensure_lds_limit(reinterpret_cast<const void*>(kern), static_cast<int>(small_lds<TT>()));
  if (e != hipSuccess) return e;
  SmallArrival arrival = {};
  float* partial = nullptr;
  bool second = false;
  if (slices > 1) {
    hipStreamCaptureStatus capturing = hipStreamCaptureStatusNone;
    const hipError_t asked = hipStreamIsCapturing(st, &capturing);
    if (asked != hipSuccess) return asked;
    second = capturing != hipStreamCaptureStatusNone;
    arrival.call = second ? 0 : call_number();
    arrival.words = static_cast<unsigned long long*>(workspace);
    partial = static_cast<float*>(workspace) + word_floats(blocks, slices);
  }
  kern<<<dim3(static_cast<uint32_t>(blocks * slices)), dim3(kSmallWaves * kWave), small_lds<TT>(), st>>>(
      p, epi, static_cast<int>(blocks), slices, static_cast<int>(steps), partial, arrival);
  const hipError_t launched = hipGetLastError();
  if (!second || launched != hipSuccess) return launched;
  small_slices_kernel<TT, Epi><<<dim3(static_cast<uint32_t>(blocks)), dim3(kSmallWaves * kWave), 0, st>>>(
      epi, static_cast<int>(p.M), p.N, slices, partial);
  return hipGetLastError();
}

template <typename E, class Epi>
hipError_t run(const Product& p, const Epi& epi, void* workspace, hipStream_t st) {
  switch (row_tiles(p.M)) {
    case 1: return launch<E, 1>(p, epi, workspace, st);
    case 2: return launch<E, 2>(p, epi, workspace, st);
    default: return launch<E, 4>(p, epi, workspace, st);
  }
}

template <typename E>
hipError_t run_type(const Product& p, void* workspace, hipStream_t st) {
  if (p.pair == kPairColumns) return run<E>(p, GatedEpilogue<E>{p.e}, workspace, st);
  if constexpr (sizeof(E) == 2) {
    if (p.out_bf16) return run<E>(p, LinearEpilogue<E, uint16_t>{p.e}, workspace, st);
  }
  return run<E>(p, LinearEpilogue<E, float>{p.e}, workspace, st);
}

}  // namespace

unsigned long long call_number() {
  static std::atomic<unsigned long long> next{
      static_cast<unsigned long long>(
          std::chrono::system_clock::now().time_since_epoch().count()) *
      0x9E3779B97F4A7C15ull};
  const unsigned long long n = next.fetch_add(1);
  return n ? n : next.fetch_add(1);
}

bool small_product(const Product& p) {
  return p.kind == kProductNN && p.M <= kSmallRows && p.K < (int64_t(1) << 31) - kSmallStep;
}

size_t small_workspace(const Product& p) {
  const int s = slices_of(p);
  if (s <= 1) return 0;
  const int64_t blocks = col_blocks(p);
  const int64_t part = int64_t(p.pair == kPairColumns ? 2 : 1) * row_tiles(p.M) * 16 * kSmallCols;
  return size_t(word_floats(blocks, s) + blocks * s * part) * sizeof(float);
}

hipError_t launch_small(const Product& p, void* workspace, hipStream_t st) {
  return p.bf16 ? run_type<uint16_t>(p, workspace, st) : run_type<float>(p, workspace, st);
}

}  // namespace fff
