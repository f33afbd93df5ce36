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
  // a NaN's rounding could carry into infinity
  static __device__ __forceinline__ T put(float f) { return f != f ? static_cast<T>(0x7FC0) : f32_to_bf16_rne(f); }
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

// Eight elements at any element's address, as float32 and back.
template <int kType>
__device__ __forceinline__ void get8(const typename Elem<kType>::T* p, float* f) {
  if constexpr (kType == QLORA_F32) {
    const u32x4 a = ld16_any(p), b = ld16_any(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = __uint_as_float(a[e]);
      f[4 + e] = __uint_as_float(b[e]);
    }
  } else {
    const u32x4 a = ld16_any(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = lo16<kType == QLORA_F16>(a[e]);
      f[2 * e + 1] = hi16<kType == QLORA_F16>(a[e]);
    }
  }
}

// Four float32 as elements, in the words [0, sizeof(T)) of a store.
template <int kType>
__device__ __forceinline__ void put4(uint32_t* w, const float* f) {
  typedef Elem<kType> E;
  if constexpr (kType == QLORA_F32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(f[e]);
  } else {
    w[0] = E::put(f[0]) | static_cast<uint32_t>(E::put(f[1])) << 16;
    w[1] = E::put(f[2]) | static_cast<uint32_t>(E::put(f[3])) << 16;
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
