// Host-side launchers of the dense feed-forward kernels: matrix products with
// an epilogue, the elementwise part of their backward passes, and activation
// checkpoints in 8 bits.  Each enqueues its kernel(s) on `st` and returns
// hipGetLastError().  Arguments have been validated by the C-ABI layer before
// any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fff {

// C[M,N] = A . B over K.  An operand is held with K contiguous in its rows,
// or k-major (row k holds consecutive rows of A or columns of B).
enum ProductKind {
  kProductNN,  // A rows, B k-major:     x . W
  kProductNT,  // A rows, B rows:        da . W^T
  kProductTN,  // A k-major, B k-major:  x^T . da
};

// Products with two B operands of the same sizes.
enum ProductPair {
  kSingle,
  kPairColumns,  // A . B0 and A . B1 in one workgroup: the gated pair
  kPairSum,      // A . B0 + (A + a_second) . B1: the gated pair's dx
  kPairTwo,      // A . B0 and A . B1 as products of their own: its weights' gradients
};

// What becomes of 32-bit sums v (and, of the gated pair, w).
struct Epilogue {
  int64_t M;
  int N;
  int act;              // fff_act_t
  const void* bias;     // layer type [N], or null
  const void* residual;  // output type [M,N], or null
  void* out[2];         // [M,N]; the second one of kPairTwo
  void* save[2];        // [M,N] v and w as they are before the activation, or null
  float* scale[2];      // [M, groups] of 8-bit saves; null: saved in the layer's type
  int group;            // columns of a scale
};

// A float32 matrix as three bf16 planes, the value being their sum: high
// (nearest), middle (the rest's nearest) and low.  Rows are padded with zeros
// to whole 16-byte pieces.
struct Planes {
  void* at;       // null: none
  int64_t ld;     // elements from a row to the next
  int64_t plane;  // elements from a plane to the next
};
inline int64_t planes_ld(int64_t cols) { return (cols + 7) / 8 * 8; }
inline size_t planes_bytes(int64_t rows, int64_t cols) {
  return 3 * size_t(rows) * size_t(planes_ld(cols)) * 2;
}

// A word that holds the call's number once a value was met that planes do not
// take: one that is not finite, or of 2^47 or more in size.
struct BeyondPlanes {
  unsigned long long* word;  // null: not asked
  unsigned long long call;
};
unsigned long long call_number();  // one that no other call has
// The word at `at` for a call on `st`, ahead of the launches that write it.
// A captured call's number may be there from a replay before that met such a
// value, so there a launch clears it: 4.5 us a replay (2048 x 1024 x 2048 93 us
// instead of 89, 8191 x 767 x 2045 162 instead of 157.5).
hipError_t start_word(void* at, hipStream_t st, BeyondPlanes& out);

struct Product {
  ProductKind kind;
  ProductPair pair;
  bool bf16;      // A, B, bias and saves; else float32
  bool out_bf16;  // out and residual
  const void *a, *b[2];
  int64_t lda, ldb;    // elements from a row to the next
  int64_t a_second;    // kPairSum: elements from A to the second segment's A
  int64_t M;
  int N;
  int64_t K;      // of one product
  Epilogue e;
  // float32 operands in planes (split_wanted), and whether one has a value beyond
  // them: the kernel on planes runs if none has, else the other one.  at of both
  // pairs' planes; the second A's follow the first's a_planes_second later.
  Planes a_planes, b_planes[2];
  int64_t a_planes_second;
  BeyondPlanes bad;
  bool padded;  // bf16: the rows have zeros up to whole 16-byte pieces
};

// Whether a float32 product is worth its operands' split into planes.
bool split_wanted(const Product& p);
// x, rows of ld floats, cols of them there, into planes.
hipError_t launch_split(const void* x, int64_t rows, int64_t cols, int64_t ld, const Planes& out,
                        const BeyondPlanes& bad, hipStream_t st);

// Whether its tiles fit one launch.
bool product_fits(const Product& p);
// Workspace of a product: its partial sums where it is cut along K.
size_t product_workspace(const Product& p);
hipError_t launch_product(const Product& p, void* workspace, hipStream_t st);

// An x kept in 8 bits, read back.
struct Restore {
  int64_t T;
  int d, group;
  const void* codes;
  const float* scale;
  void* x;     // null: none
  int64_t ld;  // elements from a row of x to the next
};

// Elementwise part of the backward passes, column sums, and the x they need,
// in one launch (and one more for the column sums' last step).
struct ActBackward {
  int64_t T;
  int N;
  bool bf16;
  bool gated;
  int act;
  const void* dy;         // [T,N]
  const void* save[2];    // pre-activation (gated: gate, up), or null where act is none
  const float* scale[2];  // of 8-bit saves, or null
  int group;
  void* da;               // [T] rows of da_ld elements, zeros behind the N; gated: the gate's,
                          // then up's; or null
  int64_t da_ld;
  void* h;                // gated: act(gate) * up [T,N], or null
  float* dbias;           // [N] sums over rows of da, or null
  float* partial;         // workspace of dbias
  Planes da_planes[2];    // float32: da (gated: the gate's and up's) once more in planes, or none
  BeyondPlanes bad;
  Restore x;
};
size_t act_backward_partials(int64_t T, int N, bool bf16);  // floats
hipError_t launch_act_backward(const ActBackward& a, hipStream_t st);

hipError_t launch_checkpoint_save(int64_t T, int d, bool bf16, int group, const void* x, void* codes,
                                  float* scale, hipStream_t st);
hipError_t launch_checkpoint_load(int64_t T, int d, bool bf16, int group, const void* codes,
                                  const float* scale, void* x, hipStream_t st);

}  // namespace fff
