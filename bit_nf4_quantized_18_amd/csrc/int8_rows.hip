// 8-bit rows: int8 codes with one float32 scale a row, made from 16- or
// 32-bit rows (the merged weight by channel, activations by token) or by the
// root-mean-square norm with the residual's addition, and turned back.
//
// For a row v with largest magnitude a: scale = fl32(a / 127), code = 127 v / a
// rounded to the nearest integer (ties to even) in exact arithmetic. The norm
// y = v rstd (v = h gain) keeps its factor rstd = 1 / sqrt(mean(h^2) + eps) out
// of the codes: 127 y / max|y| = 127 v / max|v|. It enters the scale alone, so
// both statistics of a row, sum h^2 and max|v|, come from one pass over it.
#include "elem.h"

namespace qlora {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;

// |v| as an integer: ordered as the magnitudes are, NaN above infinity, so an
// integer maximum carries a NaN through.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The code of v in a row of largest magnitude a > 0, inv = fl32(127 / a).
// t = v inv is within 127 2^-23 < 2^-15 of 127 v / a, so it rounds as that does
// unless it lies nearer than 2^-14 to a tie; the quotient in 64 bits decides
// there (127 v is exact, and a quotient that is no tie differs from one by at
// least 2^-26, far over the division's rounding). Rows so small that 127 / a
// leaves the normal range take the quotient everywhere.
__device__ __forceinline__ int encode(float v, float a, float inv) {
  const float t = v * inv;
  float c = rintf(t);
  if (fabsf(fabsf(t - c) - 0.5f) < 0x1p-14f || !(inv < 0x1p100f))
    c = static_cast<float>(rint(static_cast<double>(v) * 127.0 / static_cast<double>(a)));
  return static_cast<int>(c);
}

__device__ __forceinline__ double shfl_xor_f64(double v, int mask) { return __shfl_xor(v, mask, 64); }

// Maximum and sum over the workgroup, in every thread, in a fixed order.
__device__ __forceinline__ void reduce_row(uint32_t& top, double& sum) {
  __shared__ uint32_t tops[16];
  __shared__ double sums[16];
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    const uint32_t o = __shfl_xor(top, s, 64);
    top = o > top ? o : top;
    sum += shfl_xor_f64(sum, s);
  }
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  __syncthreads();  // the last row's values have been read
  if ((threadIdx.x & 63) == 0) {
    tops[wave] = top;
    sums[wave] = sum;
  }
  __syncthreads();
  top = tops[0];
  sum = sums[0];
  for (int i = 1; i < waves; ++i) {
    top = tops[i] > top ? tops[i] : top;
    sum += sums[i];
  }
}

struct RowArgs {
  const void* x;
  const void* residual;  // norm: may be null
  const void* gain;      // norm
  void* residual_out;    // with a residual; may be residual or x
  int64_t rows, cols, ld;
  float eps;
  int8_t* codes;
  float* scale;
};

// One workgroup a row at a time; the row is read twice, the second time from
// the cache. Every element is read and written by one thread in both passes,
// so residual_out may be one of the inputs.
template <int kType, bool kNorm, bool kGainF32>
__global__ __launch_bounds__(256) void rows_kernel(RowArgs g) {
  typedef Elem<kType> E;
  typedef typename E::T T;
  const T* gain16 = static_cast<const T*>(g.gain);
  const float* gain32 = static_cast<const float*>(g.gain);
  for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(g.x) + row * g.cols;
    const T* res = g.residual != nullptr ? static_cast<const T*>(g.residual) + row * g.cols : nullptr;
    T* out = g.residual != nullptr ? static_cast<T*>(g.residual_out) + row * g.cols : nullptr;
    uint32_t top = 0;
    double sum = 0.0;
    for (int64_t j = threadIdx.x; j < g.cols; j += blockDim.x) {
      float v = E::get(x[j]);
      if (kNorm) {
        if (res != nullptr) v += E::get(res[j]);
        sum += static_cast<double>(v) * static_cast<double>(v);
        v *= kGainF32 ? gain32[j] : E::get(gain16[j]);
      }
      const uint32_t b = mag_bits(v);
      top = b > top ? b : top;
    }
    reduce_row(top, sum);
    // a row with a NaN or an infinity: sum is not finite where h is not
    const bool bad = top >= kInfBits || !(sum < __longlong_as_double(0x7FF0000000000000LL));
    const float a = __uint_as_float(top);
    const float inv = 127.0f / a;
    if (threadIdx.x == 0) {
      double s = static_cast<double>(a) / 127.0;
      if (kNorm) s = s / sqrt(sum / static_cast<double>(g.cols) + static_cast<double>(g.eps));
      g.scale[row] = bad ? __uint_as_float(0x7FC00000u) : (top == 0 ? 0.0f : static_cast<float>(s));
    }
    const bool live = !bad && top != 0;
    int8_t* codes = g.codes + row * g.ld;
    for (int64_t j = threadIdx.x; j < g.ld; j += blockDim.x) {
      int code = 0;
      if (j < g.cols) {
        float v = E::get(x[j]);
        if (kNorm) {
          if (res != nullptr) {
            v += E::get(res[j]);
            out[j] = E::put(v);
          }
          v *= kGainF32 ? gain32[j] : E::get(gain16[j]);
        }
        if (live) code = encode(v, a, inv);
      }
      codes[j] = static_cast<int8_t>(code);
    }
  }
}

template <int kType>
__global__ __launch_bounds__(256) void dequantize_rows_kernel(const int8_t* codes, int64_t ld, const float* scale,
                                                              int64_t rows, int64_t cols, void* out) {
  typedef Elem<kType> E;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float s = scale[row];
    typename E::T* o = static_cast<typename E::T*>(out) + row * cols;
    for (int64_t j = threadIdx.x; j < cols; j += blockDim.x)
      o[j] = E::put(static_cast<float>(codes[row * ld + j]) * s);
  }
}

// Workgroups of a launch over rows: one a row, at most 2^20 (the grid's work
// items are counted in 32 bits).
unsigned row_blocks(int64_t rows) { return static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20)); }

template <int kType>
hipError_t launch_rows(const RowArgs& g, bool norm, bool gain_f32, hipStream_t s) {
  const dim3 grid(row_blocks(g.rows)), block(256);
  if (!norm) {
    hipLaunchKernelGGL((rows_kernel<kType, false, true>), grid, block, 0, s, g);
  } else if (gain_f32) {
    hipLaunchKernelGGL((rows_kernel<kType, true, true>), grid, block, 0, s, g);
  } else {
    hipLaunchKernelGGL((rows_kernel<kType, true, false>), grid, block, 0, s, g);
  }
  return hipGetLastError();
}

hipError_t launch_rows(const RowArgs& g, int dtype, bool norm, bool gain_f32, hipStream_t s) {
  if (dtype == QLORA_F32) return launch_rows<QLORA_F32>(g, norm, true, s);
  return dtype == QLORA_F16 ? launch_rows<QLORA_F16>(g, norm, gain_f32, s) : launch_rows<QLORA_BF16>(g, norm, gain_f32, s);
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int8_t* codes, int64_t ld,
                                float* scale, hipStream_t s) {
  return launch_rows(RowArgs{x, nullptr, nullptr, nullptr, rows, cols, ld, 0.0f, codes, scale}, dtype, false, true, s);
}

hipError_t launch_rmsnorm_int8(const void* x, const void* residual, const void* gain, int dtype, bool gain_f32,
                               int64_t rows, int64_t cols, float eps, void* residual_out, int8_t* codes, int64_t ld,
                               float* scale, hipStream_t s) {
  return launch_rows(RowArgs{x, residual, gain, residual_out, rows, cols, ld, eps, codes, scale}, dtype, true, gain_f32,
                     s);
}

hipError_t launch_int8_dequantize(const int8_t* codes, int64_t ld, const float* scale, int64_t rows, int64_t cols,
                                  int dtype, void* out, hipStream_t s) {
  const dim3 grid(row_blocks(rows)), block(256);
  auto kern = dtype == QLORA_F32   ? dequantize_rows_kernel<QLORA_F32>
              : dtype == QLORA_F16 ? dequantize_rows_kernel<QLORA_F16>
                                   : dequantize_rows_kernel<QLORA_BF16>;
  hipLaunchKernelGGL(kern, grid, block, 0, s, codes, ld, scale, rows, cols, out);
  return hipGetLastError();
}

}  // namespace qlora
