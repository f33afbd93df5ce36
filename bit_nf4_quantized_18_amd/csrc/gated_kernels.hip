// The product of the gated feed-forward block alone, and its gradient:
//   P = act(G) U,   dG = dP U act'(G),   dU = dP act(G),
// from the pre-activations [G | U] of gate and up, as rows of 2 n elements or as
// 8-bit rows (row 2 i the gate of token i, row 2 i + 1 its up).
//
// Element by element, so bound by memory: n elements of a token read 2 n (4 n of
// 16 bits) bytes of pre-activations, the gradient also dP, and write P or 2 n
// gradients. A thread takes kRuns runs of eight columns, all of whose loads are
// issued before the first is waited for; a run that the row's end cuts goes
// element by element. Measured: the product of 2048 x 11008 from 8-bit rows 21.6 us
// (4.2 TB/s), the gradient of 4096 x 22016 from them 126 us (5.7 TB/s); from bf16 rows
// 24 us (5.6) and 166 (5.5), from float32 46 (5.9) and 340 (5.3). The gradient of 37 x
// 5001 in float32 5.0 us, nearly all of it start and end.
#include "elem.h"
#include "gate.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

struct GatedArgs {
  const void* y;       // rows x 2 n, or
  const int8_t* codes; // 2 rows x ld with
  const float* scale;  // 2 rows scales
  const void* dp;      // backward: rows x n
  void* out;           // rows x n; backward: rows x 2 n
  uint32_t rows;       // of this launch
  int64_t n, ld;
  uint32_t chunks;     // runs of eight columns in a row
  int act;
};

// Eight 8-bit values of a row from its padded codes.
__device__ __forceinline__ void row8(u32x2 c, float s, float* f) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(static_cast<int8_t>(c[e >> 2] >> (8 * (e & 3)))) * s;
}

// One run: `row`'s columns j .. j + 7, of which `left` exist.
template <int kType, bool kRows, bool kBack>
struct Run {
  typedef typename Elem<kType>::T T;
  Words8<kType> gw, uw, dw;
  u32x2 gc, uc;
  float gs, us;
  int64_t row, j;
  int left;  // <= 0: none, < 8: the row's end cuts it

  __device__ __forceinline__ void load(const GatedArgs& g, uint32_t at, uint32_t total) {
    const uint32_t r = at / g.chunks;
    row = r;
    j = 8 * static_cast<int64_t>(at - r * g.chunks);
    left = at < total ? static_cast<int>(g.n - j < 8 ? g.n - j : 8) : 0;
    if (left <= 0) return;
    if (kRows) {  // padded rows: whole runs
      gc = *reinterpret_cast<const u32x2*>(g.codes + 2 * row * g.ld + j);
      uc = *reinterpret_cast<const u32x2*>(g.codes + (2 * row + 1) * g.ld + j);
      gs = g.scale[2 * row];
      us = g.scale[2 * row + 1];
    } else if (left == 8) {
      const T* y = static_cast<const T*>(g.y) + row * 2 * g.n + j;
      gw = load8<kType>(y);
      uw = load8<kType>(y + g.n);
    }
    if (kBack && left == 8) dw = load8<kType>(static_cast<const T*>(g.dp) + row * g.n + j);
  }

  __device__ __forceinline__ void store(const GatedArgs& g) const {
    if (left <= 0) return;
    constexpr bool kFine = kType == QLORA_F32;
    float a[8], u[8], d[8];
    const T* y = static_cast<const T*>(g.y) + row * 2 * g.n + j;
    const T* dp = static_cast<const T*>(g.dp) + row * g.n + j;
    if (kRows) {
      row8(gc, gs, a);
      row8(uc, us, u);
    } else if (left == 8) {
      values8<kType>(gw, a);
      values8<kType>(uw, u);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = e < left ? Elem<kType>::get(y[e]) : 0.0f;
        u[e] = e < left ? Elem<kType>::get(y[g.n + e]) : 0.0f;
      }
    }
    if (kBack) {
      if (left == 8) {
        values8<kType>(dw, d);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = e < left ? Elem<kType>::get(dp[e]) : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float slope;
        const float v = act_both<kFine>(a[e], g.act, &slope);
        // |slope| < 1.13: halved next to float32's end, where U act' may pass it and the
        // result need not
        const bool far = fabsf(u[e]) > 0x1p127f;
        const float part = d[e] * (u[e] * (far ? 0.5f * slope : slope));
        a[e] = far ? 2.0f * part : part;
        u[e] = d[e] * v;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = act_value<kFine>(a[e], g.act) * u[e];
    }
    T* out = static_cast<T*>(g.out) + row * (kBack ? 2 : 1) * g.n + j;
    if (left == 8) {
      put8<kType>(out, a);
      if (kBack) put8<kType>(out + g.n, u);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= left) continue;
        out[e] = Elem<kType>::put(a[e]);
        if (kBack) out[g.n + e] = Elem<kType>::put(u[e]);
      }
    }
  }
};

// The gradient may take the place of the pre-activations: every element is read
// and written by one thread, and read first.
template <int kType, bool kRows, bool kBack, int kRuns>
__global__ __launch_bounds__(kThreads) void gated_kernel(GatedArgs g) {
  const uint32_t total = g.rows * g.chunks;
  Run<kType, kRows, kBack> run[kRuns];
#pragma unroll
  for (int i = 0; i < kRuns; ++i) run[i].load(g, blockIdx.x * (kRuns * kThreads) + i * kThreads + threadIdx.x, total);
#pragma unroll
  for (int i = 0; i < kRuns; ++i) run[i].store(g);
}

template <int kType, bool kRows, bool kBack>
hipError_t launch_gated(GatedArgs g, int64_t rows, hipStream_t s) {
  constexpr int kRuns = 2;
  constexpr int64_t kMostRuns = INT64_C(1) << 30;  // of a launch: its runs are counted in 32 bits
  const int64_t size = sizeof(typename Elem<kType>::T);
  const int64_t most = kMostRuns / g.chunks;  // n <= 2^22: at least 2^11 rows
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    GatedArgs p = g;
    p.rows = static_cast<uint32_t>(rows - r0 < most ? rows - r0 : most);
    if (kRows) {
      p.codes = g.codes + 2 * r0 * g.ld;
      p.scale = g.scale + 2 * r0;
    } else {
      p.y = static_cast<const char*>(g.y) + 2 * r0 * g.n * size;
    }
    if (kBack) p.dp = static_cast<const char*>(g.dp) + r0 * g.n * size;
    p.out = static_cast<char*>(g.out) + (kBack ? 2 : 1) * r0 * g.n * size;
    const uint32_t total = p.rows * p.chunks;
    const unsigned blocks = (total + kRuns * kThreads - 1) / (kRuns * kThreads);
    hipLaunchKernelGGL((gated_kernel<kType, kRows, kBack, kRuns>), dim3(blocks), dim3(kThreads), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int kType>
hipError_t launch_gated(const GatedArgs& g, int64_t rows, hipStream_t s) {
  if (g.codes != nullptr)
    return g.dp != nullptr ? launch_gated<kType, true, true>(g, rows, s) : launch_gated<kType, true, false>(g, rows, s);
  return g.dp != nullptr ? launch_gated<kType, false, true>(g, rows, s) : launch_gated<kType, false, false>(g, rows, s);
}

}  // namespace

hipError_t launch_gated(const void* y, const int8_t* codes, int64_t ld, const float* scale, const void* dp, int dtype,
                        int64_t rows, int64_t n, int act, void* out, hipStream_t s) {
  const GatedArgs g{y, codes, scale, dp, out, 0, n, ld, static_cast<uint32_t>((n + 7) / 8), act};
  return dtype == QLORA_F32   ? launch_gated<QLORA_F32>(g, rows, s)
         : dtype == QLORA_F16 ? launch_gated<QLORA_F16>(g, rows, s)
                              : launch_gated<QLORA_BF16>(g, rows, s);
}

}  // namespace qlora
