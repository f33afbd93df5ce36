// The 8-bit product Y = (X W^T) with one scale a token and one a channel.
//
// Codes are contracted with v_mfma_i32_16x16x64_i8 into exact 32-bit integer
// sums (k 128^2 < 2^31), so the sums do not depend on the order or the split
// of the work; the scales enter once, at the end.
#include "bufmem.h"
#include "elem.h"

namespace qlora {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// D(16x16) += A(16x64) B(64x16) on int8: lane 16 g + i holds 16 codes of row i
// of A (column i of B), contraction slots 16 g .. 16 g + 15, and D[4g + v][i],
// v = 0..3. A is fed weight rows and B tokens, so a lane ends with four
// neighbouring channels of one token.
__device__ __forceinline__ i32x4 mma8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

struct LinearArgs {
  const int8_t* w;
  const float* sw;
  const int8_t* x;
  const float* sx;
  void* y;
  int64_t m, n, k;
};

constexpr int kTM = 64, kTN = 64, kTK = 64;

// 64 tokens x 64 channels a workgroup, one wave 16 channels, straight from the
// cache; rows past the edges are read from the last row and not stored.
template <int kType>
__global__ __launch_bounds__(256) void linear_kernel(LinearArgs g) {
  typename Elem<kType>::T* y = static_cast<typename Elem<kType>::T*>(g.y);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, h = lane >> 4;
  const int64_t tiles_n = (g.n + kTN - 1) / kTN;
  const int64_t m0 = blockIdx.x / tiles_n * kTM, n0 = blockIdx.x % tiles_n * kTN + 16 * wave;
  const int64_t wr = n0 + i < g.n ? n0 + i : g.n - 1;
  const int8_t* wp = g.w + wr * g.k + 16 * h;
  const int8_t* xp[4];
  i32x4 acc[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t xr = m0 + 16 * t + i < g.m ? m0 + 16 * t + i : g.m - 1;
    xp[t] = g.x + xr * g.k + 16 * h;
    acc[t] = i32x4{0, 0, 0, 0};
  }
  for (int64_t q = 0; q < g.k; q += kTK) {
    const u32x4 a = ld16(wp + q);
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = mma8(a, ld16(xp[t] + q), acc[t]);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t m = m0 + 16 * t + i;
    if (m >= g.m) continue;
    const float s = g.sx[m];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t n = n0 + 4 * h + v;
      if (n < g.n) y[m * g.n + n] = Elem<kType>::put((static_cast<float>(acc[t][v]) * s) * g.sw[n]);
    }
  }
}

}  // namespace

size_t int8_linear_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8_linear(const int8_t* w, const float* w_scale, int64_t n, int64_t k, const int8_t* x,
                              const float* x_scale, int64_t m, int out_dtype, void* y, void*, hipStream_t s) {
  const LinearArgs g{w, w_scale, x, x_scale, y, m, n, k};
  const int64_t tiles = ((m + kTM - 1) / kTM) * ((n + kTN - 1) / kTN);
  auto kern = out_dtype == QLORA_F32   ? linear_kernel<QLORA_F32>
              : out_dtype == QLORA_F16 ? linear_kernel<QLORA_F16>
                                       : linear_kernel<QLORA_BF16>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace qlora
