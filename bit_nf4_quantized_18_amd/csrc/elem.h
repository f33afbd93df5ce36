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

}  // namespace qlora
