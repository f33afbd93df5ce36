// 8-bit rows: int8 codes with one float32 scale a row, made from 16- or
// 32-bit rows (the merged weight by channel, activations by token) or by the
// root-mean-square norm with the residual's addition, and turned back.
//
// For a row v with largest magnitude a: scale = fl32(a / 127), code = 127 v / a
// rounded to the nearest integer (ties to even) in exact arithmetic. The norm
// y = v rstd (v = h gain) keeps its factor rstd = 1 / sqrt(mean(h^2) + eps) out
// of the codes: 127 y / max|y| = 127 v / max|v|. It enters the scale alone, so
// both statistics of a row, sum h^2 and max|v|, come from one pass over it.
//
// Rows of 32 bits and the norm are bound by memory: the norm of 4096 x 8192 bf16
// with its residual moves 235 MB in 48 us (4.9 TB/s; a large copy reaches 4.7),
// quantizing 11008 x 4096 float32 225 MB in 42 us, turning it back to bf16 135 MB
// in 28 us. Quantizing 16-bit rows is not: 4096 x 8192 bf16 takes 28 us, 4096 x
// 11008 39 us (3.6 and 3.5 TB/s), 1.2 elements a picosecond, as many as of
// float32 rows, which points to the instructions an element. The norm of 777 x
// 5001 fp16 takes 7.6 us for 12 MB (632 chunks in 768 places, two barriers a row;
// 5000 columns, whose rows are aligned, 7.2). One row of 4096 takes 3.6 us, with
// the norm and the residual 4.5, most of it the launch and one memory latency.
// Rows stay in registers; what decides is that all loads of a thread are in
// flight before the first is waited for: with a branch around each load the norm
// above took 63 us.
#include "elem.h"

namespace qlora {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;

// The largest magnitude of some floats as an integer: bit patterns are ordered
// as the magnitudes are, NaN above infinity, so integer maxima carry a NaN
// through. Positive values lead as signed integers, negative ones as unsigned.
struct Top {
  int pos = 0;
  uint32_t neg = 0;
  __device__ __forceinline__ void take(float v) {
    const int b = __float_as_int(v);
    pos = b > pos ? b : pos;
    neg = static_cast<uint32_t>(b) > neg ? static_cast<uint32_t>(b) : neg;
  }
  __device__ __forceinline__ uint32_t bits() const {
    const uint32_t n = neg & 0x7FFFFFFFu, p = static_cast<uint32_t>(pos);
    return n > p ? n : p;
  }
};

// Codes of eight values of a row of largest magnitude a > 0, packed; inv =
// fl32(127 / a). t = v inv is within 127 2^-23 < 2^-15 of 127 v / a, so it
// rounds as that does unless it lies nearer than 2^-14 to a tie. There (and in
// rows so small that 127 / a leaves the normal range) the quotient in 64 bits
// decides: 127 v is exact, and with v / a = 2^e V / A (V, A whole, below 2^24) a
// quotient q that is no tie differs from one by a whole number over 2 A 2^-e,
// q / (254 V) > q 2^-32 at least, far over the division's rounding q 2^-53.
// Adding 1.5 2^23 rounds to the nearest integer, ties to even, and leaves the
// code in the low byte.
__device__ __forceinline__ u32x2 encode8(const float* v, float a, float inv) {
  constexpr float kRound = 12582912.0f;
  float c[8], off = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = v[e] * inv;
    c[e] = t + kRound;
    off = fmaxf(off, fabsf(t - (c[e] - kRound)));
  }
  if (!(off < 0.5f - 0x1p-14f && inv < 0x1p100f)) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      c[e] = static_cast<float>(rint(static_cast<double>(v[e]) * 127.0 / static_cast<double>(a))) + kRound;
  }
  u32x2 out;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(c[4 * w + 1]), __float_as_uint(c[4 * w]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(c[4 * w + 3]), __float_as_uint(c[4 * w + 2]), 0x04000C0Cu);
    out[w] = lo | hi;
  }
  return out;
}

// Maximum and sum over a wave, in every lane.
__device__ __forceinline__ void reduce_wave(uint32_t& top, double& sum) {
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    const uint32_t o = __shfl_xor(top, s, 64);
    top = o > top ? o : top;
    sum += __shfl_xor(sum, s, 64);
  }
}

// Maximum and sum over the workgroup, in every thread, in a fixed order.
__device__ __forceinline__ void reduce_block(uint32_t& top, double& sum) {
  __shared__ uint32_t tops[8];
  __shared__ double sums[8];
  reduce_wave(top, sum);
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

// What a row's statistics decide.
struct RowScale {
  float a, inv, scale;
  bool live;  // it has codes other than zero
};
template <bool kNorm>
__device__ __forceinline__ RowScale row_scale(uint32_t top, double sum, const RowArgs& g) {
  // a row with a NaN or an infinity: the sum is not finite where h is not
  const bool bad = top >= kInfBits || !(sum < __longlong_as_double(0x7FF0000000000000LL));
  RowScale r;
  r.a = __uint_as_float(top);
  r.inv = 127.0f / r.a;
  double s = static_cast<double>(r.a) / 127.0;
  if (kNorm) s = s / sqrt(sum / static_cast<double>(g.cols) + static_cast<double>(g.eps));
  r.scale = bad ? __uint_as_float(0x7FC00000u) : (top == 0 ? 0.0f : static_cast<float>(s));
  r.live = !bad && top != 0;
  return r;
}

// Eight columns of a row from j on. The words are loaded without a branch (from
// the row's last eight where j + 8 passes its end), so the loads of a thread's
// chunks are all in flight before the first is waited for; rows shorter than
// eight and the chunk that the end cuts take their elements one by one.
template <int kType>
__device__ __forceinline__ Words8<kType> load_cols(const typename Elem<kType>::T* row, int64_t j, int64_t cols) {
  if (cols < 8) return Words8<kType>{};
  return load8<kType>(row + (j + 8 <= cols ? j : cols - 8));
}
template <int kType>
__device__ __forceinline__ void cols8(const Words8<kType>& w, const typename Elem<kType>::T* row, int64_t j,
                                      int64_t cols, float* f) {
  values8<kType>(w, f);
  if (j + 8 > cols) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.0f;
    if ((cols & 7) != 0 && j < cols) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < cols) f[e] = Elem<kType>::get(row[j + e]);
    }
  }
}

// The inputs of eight columns, as loaded.
template <int kType, bool kNorm, bool kRes, bool kGainF32>
struct Chunk {
  typedef typename Elem<kType>::T T;
  static constexpr int kGain = kGainF32 ? QLORA_F32 : kType;
  typedef typename Elem<kGain>::T G;
  Words8<kType> x, r;
  Words8<kGain> w;

  __device__ __forceinline__ void load(const RowArgs& g, int64_t row, int64_t j) {
    x = load_cols<kType>(static_cast<const T*>(g.x) + row * g.cols, j, g.cols);
    if (kRes) r = load_cols<kType>(static_cast<const T*>(g.residual) + row * g.cols, j, g.cols);
    if (kNorm) w = load_cols<kGain>(static_cast<const G*>(g.gain), j, g.cols);
  }

  // v = x, or (norm) h gain with h = x + residual; adds to the row's
  // statistics, and stores h.
  __device__ __forceinline__ void values(const RowArgs& g, int64_t row, int64_t j, bool store, float* v, Top& top,
                                         double& sum) const {
    const int64_t at = row * g.cols;
    cols8<kType>(x, static_cast<const T*>(g.x) + at, j, g.cols, v);
    if (kNorm) {
      float f[8];
      if (kRes) {
        cols8<kType>(r, static_cast<const T*>(g.residual) + at, j, g.cols, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += f[e];
        if (store) {
          T* out = static_cast<T*>(g.residual_out) + at;
          if (j + 8 <= g.cols) {
            put8<kType>(out + j, v);
          } else if ((g.cols & 7) != 0 && j < g.cols) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (j + e < g.cols) out[j + e] = Elem<kType>::put(v[e]);
          }
        }
      }
      cols8<kGain>(w, static_cast<const G*>(g.gain), j, g.cols, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum += static_cast<double>(v[e]) * static_cast<double>(v[e]);
        v[e] *= f[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top.take(v[e]);
  }
};

// A row in registers: thread t of the row's T threads holds columns 8 (t + i T)
// .. + 7 for i < N, read once and written once. kWave: the row's threads are a
// wave (4 rows a workgroup, no barrier), otherwise a workgroup. residual_out
// may be one of the inputs: a chunk is loaded by the one thread that stores it,
// in front of every store; where the row's end cuts chunks, the words loaded
// from its last eight columns are another thread's and are not used.
template <int kType, bool kNorm, bool kRes, bool kGainF32, int N, bool kWave>
__global__ __launch_bounds__(kWave ? 256 : 512) void rows_kernel(RowArgs g) {
  const int threads = kWave ? 64 : blockDim.x, t = kWave ? threadIdx.x & 63 : threadIdx.x;
  const int64_t rows_at_once = kWave ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x;
  const int64_t first = kWave ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  for (int64_t row = first; row < g.rows; row += rows_at_once) {
    Chunk<kType, kNorm, kRes, kGainF32> in[N];
#pragma unroll
    for (int i = 0; i < N; ++i) in[i].load(g, row, 8 * (t + i * threads));
    float v[N][8];
    Top most;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) in[i].values(g, row, 8 * (t + i * threads), true, v[i], most, sum);
    uint32_t top = most.bits();
    if (kWave) reduce_wave(top, sum);
    else reduce_block(top, sum);
    const RowScale r = row_scale<kNorm>(top, sum, g);
    if (t == 0) g.scale[row] = r.scale;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t j = 8 * (t + i * threads);
      if (j < g.ld)
        *reinterpret_cast<u32x2*>(g.codes + row * g.ld + j) = r.live ? encode8(v[i], r.a, r.inv) : u32x2{0, 0};
    }
  }
}

// Rows too long for the registers are read twice, two chunks of a thread at a
// time. Every element is read and written by one thread in both passes and h is
// stored in the second, so residual_out may be one of the inputs.
template <int kType, bool kNorm, bool kRes, bool kGainF32>
__global__ __launch_bounds__(512) void long_rows_kernel(RowArgs g) {
  const int64_t step = 8 * static_cast<int64_t>(blockDim.x);
  for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
    Top most, unused_top;
    double sum = 0.0, unused_sum = 0.0;
    float v[2][8];
    Chunk<kType, kNorm, kRes, kGainF32> in[2];
    for (int64_t j = 8 * threadIdx.x; j < g.ld; j += 2 * step) {
#pragma unroll
      for (int i = 0; i < 2; ++i) in[i].load(g, row, j + i * step);
#pragma unroll
      for (int i = 0; i < 2; ++i) in[i].values(g, row, j + i * step, false, v[i], most, sum);
    }
    uint32_t top = most.bits();
    reduce_block(top, sum);
    const RowScale r = row_scale<kNorm>(top, sum, g);
    if (threadIdx.x == 0) g.scale[row] = r.scale;
    for (int64_t j = 8 * threadIdx.x; j < g.ld; j += 2 * step) {
#pragma unroll
      for (int i = 0; i < 2; ++i) in[i].load(g, row, j + i * step);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        in[i].values(g, row, j + i * step, true, v[i], unused_top, unused_sum);
        if (j + i * step < g.ld)
          *reinterpret_cast<u32x2*>(g.codes + row * g.ld + j + i * step) =
              r.live ? encode8(v[i], r.a, r.inv) : u32x2{0, 0};
      }
    }
  }
}

// R runs of eight codes a thread; blockIdx.y takes a part of the columns.
template <int kType, int R>
__global__ __launch_bounds__(256) void dequantize_rows_kernel(const int8_t* codes, int64_t ld, const float* scale,
                                                              int64_t rows, int64_t cols, void* out, int tx) {
  typedef typename Elem<kType>::T T;
  const int64_t row_step = 256 / tx * static_cast<int64_t>(gridDim.x), step = 8 * static_cast<int64_t>(tx);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / tx) + threadIdx.x / tx; row < rows; row += row_step) {
    const float s = scale[row];
    T* o = static_cast<T*>(out) + row * cols;
    for (int64_t j0 = 8 * (threadIdx.x % tx) + R * step * blockIdx.y; j0 < cols; j0 += R * step * gridDim.y) {
      u32x2 c[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t j = j0 + i * step;
        c[i] = *reinterpret_cast<const u32x2*>(codes + row * ld + (j < ld ? j : ld - 8));
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t j = j0 + i * step;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(static_cast<int8_t>(c[i][e >> 2] >> (8 * (e & 3)))) * s;
        if (j + 8 <= cols) {
          put8<kType>(o + j, f);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (j + e < cols) o[j + e] = Elem<kType>::put(f[e]);
        }
      }
    }
  }
}

constexpr int kMaxBlocks = 1 << 20;  // a grid's work items are counted in 32 bits

unsigned blocks_for(int64_t rows, int per_block) {
  const int64_t b = (rows + per_block - 1) / per_block;
  return static_cast<unsigned>(b < kMaxBlocks ? b : kMaxBlocks);
}

template <int kType, bool kNorm, bool kRes, bool kGainF32>
hipError_t launch_rows(const RowArgs& g, hipStream_t s) {
  const int64_t chunks = g.ld / 8;
  if (chunks <= 128) {
    auto kern = chunks <= 64 ? rows_kernel<kType, kNorm, kRes, kGainF32, 1, true>
                             : rows_kernel<kType, kNorm, kRes, kGainF32, 2, true>;
    hipLaunchKernelGGL(kern, dim3(blocks_for(g.rows, 4)), dim3(256), 0, s, g);
  } else if (chunks <= 512 * 6) {
    // Few rows: as many threads as there are chunks. Many: 256 threads of up to
    // 4 chunks (2 of float32) each where these hold the row.
    const int most = g.rows <= 512 ? 1 : kType == QLORA_F32 ? 2 : 4;
    const int threads = chunks <= 256 * most ? 256 : 512;
    const int n = static_cast<int>((chunks + threads - 1) / threads);
    auto kern = n == 1   ? rows_kernel<kType, kNorm, kRes, kGainF32, 1, false>
                : n == 2 ? rows_kernel<kType, kNorm, kRes, kGainF32, 2, false>
                : n == 3 ? rows_kernel<kType, kNorm, kRes, kGainF32, 3, false>
                : n == 4 ? rows_kernel<kType, kNorm, kRes, kGainF32, 4, false>
                         : rows_kernel<kType, kNorm, kRes, kGainF32, 6, false>;
    hipLaunchKernelGGL(kern, dim3(blocks_for(g.rows, 1)), dim3(threads), 0, s, g);
  } else {
    hipLaunchKernelGGL((long_rows_kernel<kType, kNorm, kRes, kGainF32>), dim3(blocks_for(g.rows, 1)), dim3(512), 0, s,
                       g);
  }
  return hipGetLastError();
}

template <int kType>
hipError_t launch_norm(const RowArgs& g, bool gain_f32, hipStream_t s) {
  const bool res = g.residual != nullptr;
  if (kType == QLORA_F32 || gain_f32)
    return res ? launch_rows<kType, true, true, true>(g, s) : launch_rows<kType, true, false, true>(g, s);
  return res ? launch_rows<kType, true, true, false>(g, s) : launch_rows<kType, true, false, false>(g, s);
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int8_t* codes, int64_t ld,
                                float* scale, hipStream_t s) {
  const RowArgs g{x, nullptr, nullptr, nullptr, rows, cols, ld, 0.0f, codes, scale};
  return dtype == QLORA_F32   ? launch_rows<QLORA_F32, false, false, true>(g, s)
         : dtype == QLORA_F16 ? launch_rows<QLORA_F16, false, false, true>(g, s)
                              : launch_rows<QLORA_BF16, false, false, true>(g, s);
}

hipError_t launch_rmsnorm_int8(const void* x, const void* residual, const void* gain, int dtype, bool gain_f32,
                               int64_t rows, int64_t cols, float eps, void* residual_out, int8_t* codes, int64_t ld,
                               float* scale, hipStream_t s) {
  const RowArgs g{x, residual, gain, residual_out, rows, cols, ld, eps, codes, scale};
  return dtype == QLORA_F32   ? launch_norm<QLORA_F32>(g, gain_f32, s)
         : dtype == QLORA_F16 ? launch_norm<QLORA_F16>(g, gain_f32, s)
                              : launch_norm<QLORA_BF16>(g, gain_f32, s);
}

hipError_t launch_int8_dequantize(const int8_t* codes, int64_t ld, const float* scale, int64_t rows, int64_t cols,
                                  int dtype, void* out, hipStream_t s) {
  const int64_t chunks = (cols + 7) / 8;
  int tx = 8;
  while (tx < 256 && tx < chunks) tx *= 2;
  const int runs = chunks <= tx ? 1 : 4;
  const int64_t parts = (chunks + runs * tx - 1) / (runs * tx);
  const dim3 grid(blocks_for(rows, 256 / tx), static_cast<unsigned>(parts < 1024 ? parts : 1024)), block(256);
  auto kern = dtype == QLORA_F32   ? (runs == 1 ? dequantize_rows_kernel<QLORA_F32, 1> : dequantize_rows_kernel<QLORA_F32, 4>)
              : dtype == QLORA_F16 ? (runs == 1 ? dequantize_rows_kernel<QLORA_F16, 1> : dequantize_rows_kernel<QLORA_F16, 4>)
                                   : (runs == 1 ? dequantize_rows_kernel<QLORA_BF16, 1> : dequantize_rows_kernel<QLORA_BF16, 4>);
  hipLaunchKernelGGL(kern, grid, block, 0, s, codes, ld, scale, rows, cols, out, tx);
  return hipGetLastError();
}

}  // namespace qlora
