// The activations of the gated feed-forward block, act(g) = g sigma(z(g)):
//   QLORA_ACT_SILU       z = g
//   QLORA_ACT_GELU_TANH  z = 2 c (g + 0.044715 g^3), c = sqrt(2 / pi), which is
//                        0.5 g (1 + tanh(c (g + 0.044715 g^3)))
// and act'(g) = sigma + g sigma (1 - sigma) z'(g), in float32. A NaN gate gives
// NaN, an infinite one the limits: act(-inf) = -0, act' = 0; act(inf) = inf,
// act' = 1.
#pragma once

#include "internal.h"

namespace qlora {

constexpr float kGeluC = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluC3 = 0.0713548162726009f;  // 0.044715 of it

// sigma = 1 / (1 + e^-z) and 1 - sigma.
struct Sigma {
  float s, rest;
};

// kFine, for results that stay in float32: with the library's exponential of -|z| and a
// correctly rounded quotient, both parts from positive terms alone, so that neither
// loses bits where it is small, down to float32's least value. Otherwise the hardware's
// exponent and reciprocal, whose relative error, below 2^-21 (1 + |z|), vanishes in a
// rounding to 16 bits wherever sigma is not itself below that type's range; sigma is 0
// below z = -88.7, where e^-z leaves float32, and the rest is 2^-24 off, which counts
// next to the 1 that act' tends to there.
template <bool kFine>
__device__ __forceinline__ Sigma sigma(float z) {
  if constexpr (kFine) {
    const float e = expf(-fabsf(z)), r = 1.0f / (1.0f + e), er = e * r;
    return z >= 0.0f ? Sigma{r, er} : Sigma{er, r};
  } else {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
    return Sigma{s, 1.0f - s};
  }
}

template <bool kFine>
__device__ __forceinline__ float act_value(float g, int act) {
  const float z = act == QLORA_ACT_SILU ? g : g * fmaf(kGeluC3 * g, g, kGeluC);
  return fmaxf(g, -128.0f) * sigma<kFine>(z).s;  // sigma is 0 from there on: g = -inf gives no inf 0
}

// act(g) and act'(g). Beyond |g| = 128 the second term of act' is 0 in float32
// for both activations, and a gate held there keeps g^2 from overflowing.
template <bool kFine>
__device__ __forceinline__ float act_both(float g, int act, float* slope) {
  const float t = __builtin_amdgcn_fmed3f(g, -128.0f, 128.0f);
  float z = g, zs = t;
  if (act != QLORA_ACT_SILU) {
    z = g * fmaf(kGeluC3 * g, g, kGeluC);
    zs = t * fmaf(3.0f * kGeluC3 * t, t, kGeluC);
  }
  const Sigma v = sigma<kFine>(z);
  *slope = fmaf(zs * v.rest, v.s, v.s);
  return fmaxf(g, -128.0f) * v.s;
}

}  // namespace qlora
