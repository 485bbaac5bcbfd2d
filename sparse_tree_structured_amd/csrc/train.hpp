// Device helpers shared by the kernels around the layer (norm, optimiser):
// eight consecutive elements per lane, reductions over lanes, e4m3.
#pragma once

#include "common.hpp"

namespace fff {

// Eight elements move as 16-byte pieces.  The declared alignment is one
// element's: gfx950 takes unaligned global vector accesses, so rows of any
// width and tensors that start anywhere in a buffer use the same loads.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x4_t u32x4_a4_t __attribute__((aligned(4)));
typedef u32x4_t u32x4_a2_t __attribute__((aligned(2)));
typedef u32x2_t u32x2_a1_t __attribute__((aligned(1)));

// Eight elements as loaded, kept raw until they are used (half the registers
// for bf16).
template <typename E> struct Eight;

template <> struct Eight<float> {
  u32x4_t q[2];
  __device__ __forceinline__ void load(const float* p) {
    q[0] = *reinterpret_cast<const u32x4_a4_t*>(p);
    q[1] = *reinterpret_cast<const u32x4_a4_t*>(p + 4);
  }
  __device__ __forceinline__ void load_part(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i >> 2][i & 3] = i < n ? __float_as_uint(p[i]) : 0u;
  }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(q[i >> 2][i & 3]); }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    u32x4_t a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = __float_as_uint(v[i]);
      b[i] = __float_as_uint(v[4 + i]);
    }
    *reinterpret_cast<u32x4_a4_t*>(p) = a;
    *reinterpret_cast<u32x4_a4_t*>(p + 4) = b;
  }
};

template <> struct Eight<uint16_t> {
  u32x4_t q;
  __device__ __forceinline__ void load(const uint16_t* p) {
    q = *reinterpret_cast<const u32x4_a2_t*>(p);
  }
  __device__ __forceinline__ void load_part(const uint16_t* p, int n) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = e[2 * i] | (e[2 * i + 1] << 16);
  }
  __device__ __forceinline__ float get(int i) const {
    return (i & 1) ? bf16hi(q[i >> 1]) : bf16lo(q[i >> 1]);
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&v)[8]) {
    u32x4_t a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4_a2_t*>(p) = a;
  }
};

// The first n (at most 8) of eight elements; lanes with n <= 0 touch nothing.
template <typename E>
__device__ __forceinline__ void load_eight(Eight<E>& r, const E* p, int n) {
  if (n >= 8)
    r.load(p);
  else
    r.load_part(p, n);
}

template <typename E>
__device__ __forceinline__ void store_eight(E* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    Eight<E>::store(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) Elem<E>::st(p, i, v[i]);
  }
}

// ---- e4m3 (OCP: 4 exponent bits, 3 mantissa bits, largest value 448) ----

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126: no scale is below it

// Eight values of at most 448 in size to e4m3, round to nearest even.
__device__ __forceinline__ u32x2_t pack_e4m3(const float (&v)[8]) {
  u32x2_t r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
    r[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], w, true);
  }
  return r;
}

// The same down or up with the probabilities that keep the mean:
// floor(|v| / step + u) step, step an e4m3 step at |v| (2^-9 below 2^-6),
// u = the high 16 bits of rnd over 2^16 (its low 16 bits must be 0).  This is
// what gfx950's v_cvt_sr_fp8_f32 does, exact for normal and subnormal results
// (compared with the formula on four million values); it replaces eleven
// operations an element.  A |v| that its scaling left a few units above 448
// stays at 448: the carry into the next step needs more than 15 units.
__device__ __forceinline__ u32x2_t pack_e4m3_stochastic(const float (&v)[8], const uint32_t (&rnd)[8]) {
  u32x2_t r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_sr_fp8_f32(v[4 * i], rnd[4 * i], 0, 0);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(v[4 * i + 1], rnd[4 * i + 1], w, 1);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(v[4 * i + 2], rnd[4 * i + 2], w, 2);
    r[i] = __builtin_amdgcn_cvt_sr_fp8_f32(v[4 * i + 3], rnd[4 * i + 3], w, 3);
  }
  return r;
}

// 32 bits to bf16 in the same way (v_cvt_sr_bf16_f32; NaN stays NaN).
__device__ __forceinline__ u32x4_t pack_bf16_stochastic(const float (&v)[8], const uint32_t (&rnd)[8]) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bf16x2_t w = {};
    w = __builtin_amdgcn_cvt_sr_bf16_f32(w, v[2 * i], rnd[2 * i], false);
    w = __builtin_amdgcn_cvt_sr_bf16_f32(w, v[2 * i + 1], rnd[2 * i + 1], true);
    r[i] = __builtin_bit_cast(uint32_t, w);
  }
  return r;
}

// The first n of eight packed elements.
__device__ __forceinline__ void store_packed(uint8_t* p, int n, u32x2_t r) {
  if (n >= 8) {
    *reinterpret_cast<u32x2_a1_t*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(r[i >> 2] >> (8 * (i & 3)));
  }
}

__device__ __forceinline__ void store_packed(uint16_t* p, int n, u32x4_t r) {
  if (n >= 8) {
    *reinterpret_cast<u32x4_a2_t*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(r[i >> 1] >> (16 * (i & 1)));
  }
}

struct EightE4m3 {
  u32x2_t q;
  __device__ __forceinline__ void load(const uint8_t* p, int n) {
    if (n >= 8) {
      q = *reinterpret_cast<const u32x2_a1_t*>(p);
    } else {
      uint32_t e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : 0u;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        q[i] = e[4 * i] | (e[4 * i + 1] << 8) | (e[4 * i + 2] << 16) | (e[4 * i + 3] << 24);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], false);
      const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], true);
      v[4 * i] = a[0];
      v[4 * i + 1] = a[1];
      v[4 * i + 2] = b[0];
      v[4 * i + 3] = b[1];
    }
  }
};

// ---- reductions over lanes ----

// One value from another lane of the same 16: DPP controls.
constexpr int kDppXor1 = 0xB1;         // quad_perm [1,0,3,2]
constexpr int kDppXor2 = 0x4E;         // quad_perm [2,3,0,1]
constexpr int kDppHalfMirror = 0x141;  // lane i of 8 takes lane 7 - i
constexpr int kDppMirror = 0x140;      // lane i of 16 takes lane 15 - i

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false);
}

// Sum over the 64 lanes; every lane gets the same total, added in the same
// order whatever the lane.  Four DPP steps join the 16 lanes of a row, the
// two permlane swaps the four rows.
__device__ __forceinline__ float wave_total(float v) {
  v += __uint_as_float(dpp<kDppXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kDppMirror>(__float_as_uint(v)));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest size as the bits of |v|: ordered as integers, so that NaN is above
// infinity and is not lost.
__device__ __forceinline__ uint32_t size_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Maximum over groups of LANES (4, 8 or 16) consecutive lanes.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = umax(v, dpp<kDppXor1>(v));
  v = umax(v, dpp<kDppXor2>(v));
  if constexpr (LANES >= 8) v = umax(v, dpp<kDppHalfMirror>(v));
  if constexpr (LANES >= 16) v = umax(v, dpp<kDppMirror>(v));
  return v;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = group_max<16>(v);
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = umax(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return umax(b[0], b[1]);
}

// The scale of a group whose largest size has these bits (NaN stays NaN).
__device__ __forceinline__ float e4m3_scale(uint32_t bits) {
  const float s = __uint_as_float(bits) * (1.0f / kE4m3Max);
  return s < kTinyScale ? kTinyScale : s;
}

}  // namespace fff
