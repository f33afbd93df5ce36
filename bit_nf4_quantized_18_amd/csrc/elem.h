// Element types of the 8-bit row, 8-bit product and gradient kernels.
#pragma once

#include "internal.h"
#include "mfma.h"

namespace qlora {

// get: the element as float32 (exact); put: float32 to the element, round to
// nearest even, NaN kept.
template <int kType>
struct Elem;
template <>
struct Elem<QLORA_BF16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(T v) { return lo16<false>(v); }
  static __device__ __forceinline__ T put(float f) { return __builtin_bit_cast(T, static_cast<__bf16>(f)); }
};
template <>
struct Elem<QLORA_F16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(T v) { return lo16<true>(v); }
  static __device__ __forceinline__ T put(float f) {
    // the value is rounded to float32 first: without this the compiler joins a
    // product and its conversion into one instruction that rounds once
    asm("" : "+v"(f));
    return to16<true>(f);
  }
};
template <>
struct Elem<QLORA_F32> {
  typedef float T;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float f) { return f; }
};

// 16 bytes at any element's address: global memory takes them in one access
// whatever the alignment.
struct __attribute__((packed, aligned(2))) Any16 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 ld16_any(const void* p) { return static_cast<const Any16*>(p)->v; }
__device__ __forceinline__ void st16_any(void* p, u32x4 v) { static_cast<Any16*>(p)->v = v; }

// Eight elements at any element's address: the words as loaded, and their
// float32 values. Kernels load all words first and convert afterwards.
template <int kType>
struct Words8 {
  u32x4 w[sizeof(typename Elem<kType>::T) / 2];
};
template <int kType>
__device__ __forceinline__ Words8<kType> load8(const typename Elem<kType>::T* p) {
  Words8<kType> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(r.w) / sizeof(r.w[0])); ++i)
    r.w[i] = ld16_any(reinterpret_cast<const char*>(p) + 16 * i);
  return r;
}
template <int kType>
__device__ __forceinline__ void values8(const Words8<kType>& r, float* f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (kType == QLORA_F32) {
      f[e] = __uint_as_float(r.w[0][e]);
      f[4 + e] = __uint_as_float(r.w[1][e]);
    } else {
      f[2 * e] = lo16<kType == QLORA_F16>(r.w[0][e]);
      f[2 * e + 1] = hi16<kType == QLORA_F16>(r.w[0][e]);
    }
  }
}

// Two float32 as a pair of 16-bit elements.
template <int kType>
__device__ __forceinline__ uint32_t put2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  if constexpr (kType == QLORA_BF16)  // one instruction on gfx950
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
  else
    return Elem<kType>::put(a) | static_cast<uint32_t>(Elem<kType>::put(b)) << 16;
}

// Four float32 as elements, in the words [0, sizeof(T)) of a store.
template <int kType>
__device__ __forceinline__ void put4(uint32_t* w, const float* f) {
  if constexpr (kType == QLORA_F32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(f[e]);
  } else {
    w[0] = put2<kType>(f[0], f[1]);
    w[1] = put2<kType>(f[2], f[3]);
  }
}

template <int kType>
__device__ __forceinline__ void put8(typename Elem<kType>::T* p, const float* f) {
  constexpr int kWords = 2 * sizeof(typename Elem<kType>::T);
  union {
    uint32_t w[kWords];
    u32x4 v[kWords / 4];
  } out;
  put4<kType>(out.w, f);
  put4<kType>(out.w + kWords / 2, f + 4);
#pragma unroll
  for (int j = 0; j < kWords / 4; ++j) st16_any(reinterpret_cast<u32x4*>(p) + j, out.v[j]);
}

}  // namespace qlora
