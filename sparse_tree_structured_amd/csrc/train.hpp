// Device helpers shared by the kernels around the layer (norm, optimiser):
// consecutive elements per lane, reductions over lanes, e4m3.
#pragma once

#include "common.hpp"

namespace fff {

// A lane moves V consecutive elements (V * sizeof(E) = 4, 8 or 16 bytes) as
// one access, so that a wavefront's access is one contiguous piece.  The
// declared alignment is one element's: gfx950 takes unaligned global vector
// accesses, so rows of any width and tensors that start anywhere in a buffer
// use the same loads.
template <int WORDS> struct WordsOf { typedef uint32_t type __attribute__((ext_vector_type(WORDS))); };
template <> struct WordsOf<1> { typedef uint32_t type; };

template <typename T, int ALIGN> struct Unaligned;
template <typename T> struct Unaligned<T, 4> { typedef T type __attribute__((aligned(4))); };
template <typename T> struct Unaligned<T, 2> { typedef T type __attribute__((aligned(2))); };
template <typename T> struct Unaligned<T, 1> { typedef T type __attribute__((aligned(1))); };

__device__ __forceinline__ uint32_t word_of(uint32_t w, int) { return w; }
template <typename T> __device__ __forceinline__ uint32_t word_of(T w, int i) { return w[i]; }
__device__ __forceinline__ void set_word(uint32_t& w, int, uint32_t v) { w = v; }
template <typename T> __device__ __forceinline__ void set_word(T& w, int i, uint32_t v) { w[i] = v; }

// V elements as they lie in memory.  STREAM: the access does not ask to stay
// in the caches.
template <typename E, int V>
struct Pack {
  static constexpr int kWords = V * int(sizeof(E)) / 4;
  static constexpr int kPer = 4 / int(sizeof(E));  // elements of a word
  static constexpr int kBits = 8 * int(sizeof(E));
  typedef typename WordsOf<kWords>::type words_t;
  typedef typename Unaligned<words_t, int(sizeof(E))>::type at_t;
  words_t q;

  __device__ __forceinline__ uint32_t word(int i) const { return word_of(q, i); }

  // The first n of V elements, the others 0 (n <= 0 touches nothing).
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const E* p, int n) {
    if (n >= V) {
      if constexpr (STREAM)
        q = __builtin_nontemporal_load(reinterpret_cast<const at_t*>(p));
      else
        q = *reinterpret_cast<const at_t*>(p);
      return;
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      uint32_t v = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (w * kPer + i < n) v |= bits_of(p[w * kPer + i]) << (kBits * i);
      set_word(q, w, v);
    }
  }

  template <bool STREAM = false>
  __device__ __forceinline__ void store(E* p, int n) const {
    if (n >= V) {
      if constexpr (STREAM)
        __builtin_nontemporal_store(q, reinterpret_cast<at_t*>(p));
      else
        *reinterpret_cast<at_t*>(p) = q;
      return;
    }
    store_range(p, 0, n);
  }

  // Elements lo .. hi - 1 of the V at p.
  __device__ __forceinline__ void store_range(E* p, int lo, int hi) const {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i >= lo && i < hi) put_bits(p + i, word(i / kPer) >> (kBits * (i % kPer)));
  }

  // As 32-bit floats (float and bf16).
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(E) == 4) return __uint_as_float(word(i));
    return (i & 1) ? bf16hi(word(i >> 1)) : bf16lo(word(i >> 1));
  }
  __device__ __forceinline__ void set(const float (&v)[V]) {
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      if constexpr (sizeof(E) == 4)
        set_word(q, w, __float_as_uint(v[w]));
      else
        set_word(q, w, pack_bf16x2(v[2 * w], v[2 * w + 1]));
    }
  }

  static __device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }
  static __device__ __forceinline__ uint32_t bits_of(uint16_t v) { return v; }
  static __device__ __forceinline__ uint32_t bits_of(uint8_t v) { return v; }
  static __device__ __forceinline__ void put_bits(float* p, uint32_t b) { *p = __uint_as_float(b); }
  static __device__ __forceinline__ void put_bits(uint16_t* p, uint32_t b) { *p = uint16_t(b); }
  static __device__ __forceinline__ void put_bits(uint8_t* p, uint32_t b) { *p = uint8_t(b); }
};

template <typename E, int V>
__device__ __forceinline__ Pack<E, V> packed(const float (&v)[V]) {
  Pack<E, V> r;
  r.set(v);
  return r;
}

// ---- e4m3 (OCP: 4 exponent bits, 3 mantissa bits, largest value 448) ----

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126: no scale is below it

// V values of at most 448 in size to e4m3, round to nearest even.
template <int V>
__device__ __forceinline__ Pack<uint8_t, V> pack_e4m3(const float (&v)[V]) {
  Pack<uint8_t, V> r;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
    set_word(r.q, i, __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], w, true));
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
template <int V>
__device__ __forceinline__ Pack<uint8_t, V> pack_e4m3_stochastic(const float (&v)[V],
                                                                 const uint32_t (&rnd)[V]) {
  Pack<uint8_t, V> r;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    int w = __builtin_amdgcn_cvt_sr_fp8_f32(v[4 * i], rnd[4 * i], 0, 0);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(v[4 * i + 1], rnd[4 * i + 1], w, 1);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(v[4 * i + 2], rnd[4 * i + 2], w, 2);
    set_word(r.q, i, __builtin_amdgcn_cvt_sr_fp8_f32(v[4 * i + 3], rnd[4 * i + 3], w, 3));
  }
  return r;
}

// 32 bits to bf16 in the same way (v_cvt_sr_bf16_f32; NaN stays NaN).
template <int V>
__device__ __forceinline__ Pack<uint16_t, V> pack_bf16_stochastic(const float (&v)[V],
                                                                  const uint32_t (&rnd)[V]) {
  Pack<uint16_t, V> r;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    bf16x2_t w = {};
    w = __builtin_amdgcn_cvt_sr_bf16_f32(w, v[2 * i], rnd[2 * i], false);
    w = __builtin_amdgcn_cvt_sr_bf16_f32(w, v[2 * i + 1], rnd[2 * i + 1], true);
    set_word(r.q, i, __builtin_bit_cast(uint32_t, w));
  }
  return r;
}

// e4m3 codes as 32-bit floats.
template <int V>
__device__ __forceinline__ void unpack_e4m3(const Pack<uint8_t, V>& r, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(r.word(i), false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(r.word(i), true);
    v[4 * i] = a[0];
    v[4 * i + 1] = a[1];
    v[4 * i + 2] = b[0];
    v[4 * i + 3] = b[1];
  }
}

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

// Maximum over groups of LANES (4, 8, 16 or 32) consecutive lanes.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = umax(v, dpp<kDppXor1>(v));
  v = umax(v, dpp<kDppXor2>(v));
  if constexpr (LANES >= 8) v = umax(v, dpp<kDppHalfMirror>(v));
  if constexpr (LANES >= 16) v = umax(v, dpp<kDppMirror>(v));
  if constexpr (LANES >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = umax(a[0], a[1]);
  }
  return v;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = group_max<32>(v);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return umax(b[0], b[1]);
}

// The scale of a group whose largest size has these bits (NaN stays NaN).
__device__ __forceinline__ float e4m3_scale(uint32_t bits) {
  const float s = __uint_as_float(bits) * (1.0f / kE4m3Max);
  return s < kTinyScale ? kTinyScale : s;
}

// 1 / s for a scale, correctly rounded: an approximation and one correction
// by fma (equal to the IEEE quotient for every s from 2^-126 to 2^120; a
// scale is at most 2^128 / 448, or infinite).
__device__ __forceinline__ float reciprocal(float s) {
#pragma clang fp contract(off)
  const float y = __builtin_amdgcn_rcpf(s);
  const float r = __builtin_fmaf(__builtin_fmaf(-s, y, 1.0f), y, y);
  return __builtin_isinf(s) ? 0.0f : r;
}

}  // namespace fff
