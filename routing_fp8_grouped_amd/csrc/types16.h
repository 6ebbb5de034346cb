// Element types of the operators whose operands are not quantised (BF16, FP16,
// FP32): 16-byte chunks of them, and conversions.
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// kWidth elements make one 16-byte chunk.  Stores round to nearest even
// (hardware conversions: infinities and NaN stay what they are).
struct Bf16 {
  using storage = uint16_t;
  using frag = v8bf;
  static constexpr int kWidth = 8;
  static __device__ __forceinline__ float load(storage s) { return bf16_to_f32(s); }
  static __device__ __forceinline__ storage store(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
  static __device__ __forceinline__ uint32_t store2(float lo, float hi) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{lo, hi}, v2bf));
  }
  static __device__ __forceinline__ v4f mfma(frag a, frag b, v4f c) { return mfma_bf16_16x16x32(a, b, c); }
};
struct Fp16 {
  using storage = uint16_t;
  using frag = v8h;
  static constexpr int kWidth = 8;
  static __device__ __forceinline__ float load(storage s) { return (float)__builtin_bit_cast(_Float16, s); }
  static __device__ __forceinline__ storage store(float f) {
    asm("" : "+v"(f));   // the FP32 value is what is rounded: no mixed-precision product straight to FP16
    return __builtin_bit_cast(uint16_t, (_Float16)f);
  }
  static __device__ __forceinline__ uint32_t store2(float lo, float hi) {
    return (uint32_t)store(lo) | ((uint32_t)store(hi) << 16);
  }
  static __device__ __forceinline__ v4f mfma(frag a, frag b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
struct Fp32 {
  using storage = float;
  static constexpr int kWidth = 4;
  static __device__ __forceinline__ float load(storage s) { return s; }
  static __device__ __forceinline__ storage store(float f) { return f; }
};

// Two values in the two halves of a word.
template <class E>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return E::store2(lo, hi);
}
template <class E>
__device__ __forceinline__ float unpack(uint32_t word, int half) {
  return E::load((uint16_t)(word >> (16 * half)));
}

// 16 bytes at an address that is only aligned to its elements (rows of any
// width): global memory takes them in one instruction all the same.  PAST: data
// that goes past the caches.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <bool PAST = false, class S>
__device__ __forceinline__ u32x4 load_chunk(const S* p) {
  const u32x4_any* q = reinterpret_cast<const u32x4_any*>(p);
  if constexpr (PAST) return __builtin_nontemporal_load(q);
  else return *q;
}
template <bool PAST = false, class S>
__device__ __forceinline__ void store_chunk(S* p, u32x4 v) {
  u32x4_any* q = reinterpret_cast<u32x4_any*>(p);
  if constexpr (PAST) __builtin_nontemporal_store(v, q);
  else *q = v;
}

// FP32 values of a 16-byte chunk (WHOLE) or of one element.
template <class E, bool WHOLE>
struct Values {
  using S = typename E::storage;
  using raw = std::conditional_t<WHOLE, u32x4, S>;
  static constexpr int n = WHOLE ? E::kWidth : 1;
  float v[n];

  template <bool PAST = false>
  static __device__ __forceinline__ raw fetch(const S* p) {
    if constexpr (WHOLE) return load_chunk<PAST>(p);
    else return *p;
  }
  __device__ __forceinline__ Values() {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ explicit Values(raw w) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if constexpr (!WHOLE) v[i] = E::load(w);
      else if constexpr (E::kWidth == 8) v[i] = unpack<E>(w[i / 2], i & 1);
      else v[i] = __uint_as_float(w[i]);
    }
  }
  template <bool PAST = false>
  __device__ __forceinline__ void put(S* p) const {
    if constexpr (WHOLE) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (E::kWidth == 8) w[i] = pack2<E>(v[2 * i], v[2 * i + 1]);
        else w[i] = __float_as_uint(v[i]);
      }
      store_chunk<PAST>(p, w);
    } else {
      *p = E::store(v[0]);
    }
  }
};

}  // namespace moe
