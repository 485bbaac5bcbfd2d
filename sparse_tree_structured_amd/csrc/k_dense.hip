// Matrix products of the dense feed-forward block: how one is cut into tiles
// and slices of K, and the sums of the slices.
#include "product.hpp"

namespace fff {
namespace {

// The slices' sums, added in their order, through the epilogue: a wavefront
// has 256 columns of a row.
template <class Epi>
__global__ __launch_bounds__(256) void sum_slices_kernel(const float* partial, int slices,
                                                         int products, int64_t M, int N, Epi epi,
                                                         BeyondPlanes bad) {
  if (bad.word && *bad.word == bad.call) return;
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

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether the rows of both operands are whole 16-byte pieces (K too: a longer
// row's rest is zeros in the workspace's da only, which cut_product is told).
bool direct_sizes(const Product& p) {
  if (p.lda % 8 != 0 || p.ldb % 8 != 0 || p.a_second % 8 != 0) return false;
  return p.kind == kProductTN || p.K % 8 == 0;
}

struct TileSize {
  ProductTile tile;
  int m, n, bk;
  double rate;  // of its matrix-core work, FLOP/s of a compute unit
  int together = 1;      // workgroups of a compute unit that hide each other's steps
  double step_us = 0.25;  // the shortest time of a step
};

// The time of a product in one kind of tile and number of slices, in us: what
// the busiest compute unit does, a start and an epilogue for each of its
// tiles, and for slices a second launch and the sums' way through memory.
// The rates are those measured on one tile's work with the chip full; that of the
// register-staged bf16 tile (1.5 us a step) is of few tiles of odd rows, where it
// decides whether to copy.  What the model chooses in bf16, as measured (us): 512 x 2048 x 1024 12.4, 1024 x 2048
// x 4096 31, 2048 x 2048 x 4096 44, 4096 x 2048 x 4096 64 (1.07 PFLOP/s).
double time_of(const Product& p, const TileSize& t, int64_t tiles, int64_t total, int64_t slices) {
  const int64_t steps = ceil_div(total, slices);
  const int64_t each = ceil_div(tiles * slices, 256);  // of the busiest compute unit
  const int64_t rounds = ceil_div(each, t.together);
  const double busy = 2.0 * t.m * t.n * t.bk / t.rate * 1e6 * (each < t.together ? each : t.together);
  double us = rounds * (steps * (busy > t.step_us ? busy : t.step_us) + 4.0);
  if (slices > 1) {
    const int products = p.pair == kPairColumns || p.pair == kPairTwo ? 2 : 1;
    us += 5.0 + 8.0 * slices * products * p.M * p.N / 4e6;
  }
  return us;
}

Cut cut_with(const Product& p, const TileSize& t, double& us) {
  Cut c;
  c.tile = t.tile;
  c.tiles_m = ceil_div(p.M, t.m);
  c.tiles_n = ceil_div(p.N, p.pair == kPairColumns ? t.n / 2 : t.n);
  c.products = p.pair == kPairColumns || p.pair == kPairTwo ? 2 : 1;
  int64_t tiles = c.tiles_m * c.tiles_n * (p.pair == kPairTwo ? 2 : 1);
  if (tiles < 1) tiles = 1;
  int64_t total = ceil_div(p.K, t.bk) * (p.pair == kPairSum ? 2 : 1);
  if (!p.bf16 && t.tile >= kTileBig) total *= 6;  // on planes
  int64_t slices = 1;
  us = time_of(p, t, tiles, total, 1);
  // Slices of at least four steps while tiles leave compute units idle.
  for (int64_t s = 2; s * tiles <= 512 * t.together && s * 4 <= total; ++s) {
    const double with = time_of(p, t, tiles, total, s);
    if (with < us) us = with, slices = s;
  }
  c.steps = static_cast<int>(ceil_div(total, slices));
  c.slices = total > 0 ? static_cast<int>(ceil_div(total, c.steps)) : 1;
  return c;
}

Cut cut_direct(const Product& p, double* us_of = nullptr) {
  static const TileSize kTiles[] = {{kTileBig, 256, 256, 64, 4.9e12},
                                    {kTileMid, 128, 256, 64, 3.6e12},
                                    {kTileSmall, 128, 128, 64, 3.2e12}};
  Cut best = {};
  double least = 0;
  for (const TileSize& t : kTiles) {
    if (t.tile == kTileSmall && p.pair == kPairColumns) continue;
    double us;
    const Cut c = cut_with(p, t, us);
    if (t.tile == kTileBig || us < least) best = c, least = us;
  }
  if (us_of) *us_of = least;
  return best;
}

Cut cut_any(const Product& p, double* us_of = nullptr) {
  double own, &us = us_of ? *us_of : own;
  Cut c = cut_with(p, {kTileAny, 128, 256, p.bf16 ? 32 : 16, p.bf16 ? 1.4e12 : 0.45e12}, us);
  // Float32 steps of the large tile take 2 us each: small products are spread
  // further (512 x 512 x 2048 33 -> 26 us, 128 x 512 x 128 20 -> 12).
  if (!p.bf16 && p.pair != kPairColumns) {
    double small;
    const Cut s = cut_with(p, {kTileAnySmall, 64, 128, 16, 0.5e12, 4, 0.95}, small);
    if (small < us) c = s, us = small;
  }
  return c;
}

// Splits of x [rows, cols] float32 into planes: a lane has eight columns, the
// row's padding among them.
__global__ __launch_bounds__(256) void split_kernel(const float* x, int64_t rows, int64_t cols, int64_t ld,
                                                    Planes out, BeyondPlanes bad) {
  const int64_t pieces = out.ld / 8;
  bool odd = false;
  for (int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x; u < rows * pieces;
       u += int64_t(gridDim.x) * 256) {
    const int64_t row = u / pieces, col = u % pieces * 8;
    float v[8];
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
      const int64_t left = cols - col - h;
      Pack<float, 4> q;
      q.load(x + row * ld + col + h, left < 4 ? static_cast<int>(left) : 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[h + i] = q.get(i);
    }
    odd |= store_planes<8>(v, static_cast<uint16_t*>(out.at) + row * out.ld + col, out.plane, 8);
  }
  if (odd) *bad.word = bad.call;
}

// (no call has the number 0)
__global__ __launch_bounds__(64) void clear_word_kernel(unsigned long long* word) {
  if (threadIdx.x == 0) *word = 0;
}

// Copies x [rows, cols] bf16 to rows of `to_ld`, zeros behind the columns.
__global__ __launch_bounds__(256) void pad_kernel(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                                                  uint16_t* to, int64_t to_ld) {
  const int64_t pieces = to_ld / 8;
  for (int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x; u < rows * pieces;
       u += int64_t(gridDim.x) * 256) {
    const int64_t row = u / pieces, col = u % pieces * 8;
    const int64_t left = cols - col;
    Pack<uint16_t, 8> q;
    q.load(x + row * ld + col, left < 8 ? static_cast<int>(left) : 8);
    q.store(to + row * to_ld + col, 8);
  }
}

hipError_t launch_pad(const void* x, int64_t rows, int64_t cols, int64_t ld, void* to, int64_t to_ld,
                      hipStream_t st) {
  const int64_t blocks = ceil_div(rows * (to_ld / 8), 256);
  pad_kernel<<<dim3(static_cast<uint32_t>(blocks < 16384 ? blocks : 16384)), dim3(256), 0, st>>>(
      static_cast<const uint16_t*>(x), rows, cols, ld, static_cast<uint16_t*>(to), to_ld);
  return hipGetLastError();
}

// Which operands of a bf16 product do not have rows of whole pieces.
struct Padding {
  bool a, b;
};
Padding padding_of(const Product& p) {
  return {p.lda % 8 != 0, p.ldb % 8 != 0};
}

// Whether the operands but those that are copied are aligned.
bool operands_aligned(const Product& p, const Padding& copied) {
  if (!copied.a && !aligned16(p.a)) return false;
  return copied.b || (aligned16(p.b[0]) && (p.pair == kSingle || aligned16(p.b[1])));
}

size_t cut_bytes(const Product& p, const Cut& c) {
  return c.slices <= 1 ? 0
                       : size_t(c.slices) * c.products * size_t(p.M) * size_t(p.N) * sizeof(float);
}

}  // namespace

template <class Epi>
hipError_t launch_sum_slices(const float* partial, const Cut& c, int64_t M, int N, const Epi& epi,
                             const BeyondPlanes& bad, hipStream_t st) {
  const int64_t units = M * ceil_div(N, 256) * (Epi::kGated ? 1 : c.products);
  const int64_t blocks = ceil_div(units, 4);
  sum_slices_kernel<Epi><<<dim3(static_cast<uint32_t>(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                           st>>>(partial, c.slices, c.products, M, N, epi, bad);
  return hipGetLastError();
}
#define FFF_SUM(E)                                                                                \
  template hipError_t launch_sum_slices<E>(const float*, const Cut&, int64_t, int, const E&, \
                                           const BeyondPlanes&, hipStream_t)
FFF_SUM(GatedEpilogue<uint16_t>);
FFF_SUM(GatedEpilogue<float>);
using LinearBf16 = LinearEpilogue<uint16_t, uint16_t>;
using LinearMixed = LinearEpilogue<uint16_t, float>;
using LinearF32 = LinearEpilogue<float, float>;
FFF_SUM(LinearBf16);
FFF_SUM(LinearMixed);
FFF_SUM(LinearF32);

Cut cut_whole(const Product& p) {
  Cut c = cut_any(p);
  c.steps *= c.slices;
  c.slices = 1;
  return c;
}

// A product on planes takes six times the bf16 one's work at its rate, the
// planes 10 bytes an element and two launches; on its values a sixteenth of
// the rate.  8191 x 767 x 2045 with GELU and 8-bit saves takes 170 us instead of
// 241, 1024 x 2048 x 2048 85 instead of 100; at 512 x 2048 x 2048 the values
// take 56.
bool split_wanted(const Product& p) {
  if (p.bf16) return false;
  const double pairs = p.pair == kSingle ? 1 : 2;
  const double flops = 2.0 * pairs * p.M * p.N * p.K;
  const double elements = double(p.M) * p.K * (p.pair == kPairSum ? 2 : 1) + pairs * p.K * p.N;
  return flops / 90e6 > 6 * flops / 1100e6 + 10 * elements / 4e6 + 20.0;
}

hipError_t launch_split(const void* x, int64_t rows, int64_t cols, int64_t ld, const Planes& out,
                        const BeyondPlanes& bad, hipStream_t st) {
  const int64_t blocks = ceil_div(rows * (out.ld / 8), 256);
  split_kernel<<<dim3(static_cast<uint32_t>(blocks < 16384 ? blocks : 16384)), dim3(256), 0, st>>>(
      static_cast<const float*>(x), rows, cols, ld, out, bad);
  return hipGetLastError();
}

hipError_t start_word(void* at, hipStream_t st, BeyondPlanes& out) {
  out = {static_cast<unsigned long long*>(at), call_number()};
  hipStreamCaptureStatus capturing = hipStreamCaptureStatusNone;
  const hipError_t asked = hipStreamIsCapturing(st, &capturing);
  if (asked != hipSuccess || capturing == hipStreamCaptureStatusNone) return asked;
  clear_word_kernel<<<dim3(1), dim3(64), 0, st>>>(out.word);
  return hipGetLastError();
}

Cut cut_product(const Product& p) {
  if (!p.bf16) return p.bad.word ? cut_direct(p) : cut_any(p);
  return p.padded || (direct_sizes(p) && operands_aligned(p, {})) ? cut_direct(p) : cut_any(p);
}

bool product_fits(const Product& p) {
  // (a launch has fewer than 2^32 threads)
  auto fits = [&](const Cut& c) {
    const int64_t threads = c.tile == kTileAnySmall || c.tile == kTileSmall ? 256 : 512;
    return c.tiles_m * c.tiles_n * c.slices * (p.pair == kPairTwo ? 2 : 1) * threads < (int64_t(1) << 32);
  };
  return fits(cut_any(p)) && fits(cut_direct(p));
}

namespace {

size_t padded(size_t bytes) { return (bytes + 255) & ~size_t(255); }

// Rows and columns of an operand as it lies in memory.
void a_sizes(const Product& p, int64_t& rows, int64_t& cols) {
  rows = p.kind == kProductTN ? p.K : p.M;
  cols = p.kind == kProductTN ? p.M : p.K;
}
void b_sizes(const Product& p, int64_t& rows, int64_t& cols) {
  rows = p.kind == kProductNT ? p.N : p.K;
  cols = p.kind == kProductNT ? p.K : p.N;
}

// Where a product on planes has what it makes: the slices' sums, a word, and
// the planes of the operands that have none yet (no row length).
struct PlanesAt {
  size_t word, a, b[2], bytes;
};
PlanesAt planes_at(const Product& p) {
  PlanesAt l = {};
  int64_t rows, cols;
  l.word = padded(cut_bytes(p, cut_direct(p)));
  l.bytes = l.word + 256;
  if (p.a_planes.ld == 0) {
    a_sizes(p, rows, cols);
    l.a = l.bytes;
    l.bytes += padded(planes_bytes(rows, cols));
  }
  b_sizes(p, rows, cols);
  for (int i = 0; i < (p.pair == kSingle ? 1 : 2); ++i)
    if (p.b_planes[i].ld == 0) {
      l.b[i] = l.bytes;
      l.bytes += padded(planes_bytes(rows, cols));
    }
  return l;
}

hipError_t split_operand(const void* x, int64_t rows, int64_t cols, int64_t ld, unsigned char* to,
                         Planes& out, const BeyondPlanes& bad, hipStream_t st) {
  out = {to, planes_ld(cols), rows * planes_ld(cols)};
  return launch_split(x, rows, cols, ld, out, bad, st);
}

// Whether copies with padded rows, for the tiles straight into LDS, are worth
// their time: 2048 x 4095 x 2047 takes 61 us instead of 137 (the gated pair 88
// instead of 245), 512 x 767 x 2045 20 instead of 23; 128 x 767 x 2045 18 either way.
bool padding_wanted(const Product& p) {
  if (!p.bf16 || p.K == 0) return false;  // (gradients of no rows: zeros, and nothing to copy)
  const Padding pad = padding_of(p);
  if (!pad.a && !pad.b) return false;
  int64_t rows, cols;
  double us = 0, direct = 0, any = 0;
  a_sizes(p, rows, cols);
  if (pad.a) us += 4.0 + 4.0 * rows * cols / 4e6;
  b_sizes(p, rows, cols);
  if (pad.b) us += (p.pair == kSingle ? 1 : 2) * (4.0 + 4.0 * rows * cols / 4e6);
  cut_direct(p, &direct);
  cut_any(p, &any);
  return us + direct < any;
}

PlanesAt padded_at(const Product& p) {
  PlanesAt l = {};
  const Padding pad = padding_of(p);
  int64_t rows, cols;
  l.bytes = padded(cut_bytes(p, cut_direct(p)));
  a_sizes(p, rows, cols);
  if (pad.a) {
    l.a = l.bytes;
    l.bytes += padded(size_t(rows) * planes_ld(cols) * 2);
  }
  b_sizes(p, rows, cols);
  for (int i = 0; pad.b && i < (p.pair == kSingle ? 1 : 2); ++i) {
    l.b[i] = l.bytes;
    l.bytes += padded(size_t(rows) * planes_ld(cols) * 2);
  }
  return l;
}


}  // namespace

// For pointers of any alignment.
size_t product_workspace(const Product& p) {
  size_t most = cut_bytes(p, cut_any(p));
  const size_t direct = !p.bf16           ? (split_wanted(p) ? planes_at(p).bytes : 0)
                        : direct_sizes(p)   ? cut_bytes(p, cut_direct(p))
                        : padding_wanted(p) ? padded_at(p).bytes
                                            : 0;
  const size_t small = small_product(p) ? small_workspace(p) : 0;
  if (direct > most) most = direct;
  return small > most ? small : most;
}

hipError_t launch_product(const Product& product, void* workspace, hipStream_t st) {
  Product p = product;
  // (a few rows' kernel has 64 columns of a row together: no groups of 128)
  const bool wide = (p.e.scale[0] || p.e.scale[1]) && p.e.group == 128;
  if (small_product(p) && !wide) {
    p.bad = {};
    return launch_small(p, workspace, st);
  }
  const Padding pad = padding_of(p);
  if (padding_wanted(p) && operands_aligned(p, pad)) {
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    const PlanesAt l = padded_at(p);
    int64_t rows, cols;
    hipError_t e = hipSuccess;
    a_sizes(p, rows, cols);
    if (pad.a) {
      e = launch_pad(p.a, rows, cols, p.lda, ws + l.a, planes_ld(cols), st);
      p.a = ws + l.a;
      p.lda = planes_ld(cols);
    }
    b_sizes(p, rows, cols);
    for (int i = 0; pad.b && i < (p.pair == kSingle ? 1 : 2) && e == hipSuccess; ++i) {
      e = launch_pad(p.b[i], rows, cols, p.ldb, ws + l.b[i], planes_ld(cols), st);
      p.b[i] = ws + l.b[i];
    }
    if (pad.b) p.ldb = planes_ld(cols);
    p.padded = true;
    if (e != hipSuccess) return e;
  }
  if (!split_wanted(p)) {
    p.bad = {};
  } else {
    unsigned char* const ws = static_cast<unsigned char*>(workspace);
    const PlanesAt l = planes_at(p);
    hipError_t e = hipSuccess;
    int64_t rows, cols;
    if (!p.bad.word) e = start_word(ws + l.word, st, p.bad);
    if (e == hipSuccess && !p.a_planes.at) {
      a_sizes(p, rows, cols);
      e = split_operand(p.a, rows, cols, p.lda, ws + l.a, p.a_planes, p.bad, st);
    }
    b_sizes(p, rows, cols);
    for (int i = 0; i < (p.pair == kSingle ? 1 : 2); ++i)
      if (e == hipSuccess && !p.b_planes[i].at)
        e = split_operand(p.b[i], rows, cols, p.ldb, ws + l.b[i], p.b_planes[i], p.bad, st);
    if (e != hipSuccess) return e;
  }
  if (p.kind == kProductNN) return run_nn(p, workspace, st);
  return p.kind == kProductNT ? run_nt(p, workspace, st) : run_tn(p, workspace, st);
}

}  // namespace fff
