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

// ---------------------------------------------------------------------------
// Tiles through LDS.
// ---------------------------------------------------------------------------
constexpr int kBK = 64;     // contraction codes a step: one MFMA deep
constexpr int kStages = 4;  // LDS ring
constexpr int kXcds = 8;

template <int BM, int BN>
constexpr int stage_bytes() {
  return (BM + BN) * kBK;
}

// 16 neighbouring outputs of one token: (acc sx) sw, each rounded once, the
// first `left` of them stored.
template <int kType>
__device__ __forceinline__ void store_run(typename Elem<kType>::T* y, const i32x4* acc, float sx, const float* sw,
                                          int64_t left) {
  constexpr int kWords = 4 * sizeof(typename Elem<kType>::T);
  union {
    uint32_t w[kWords];
    u32x4 v[kWords / 4];
    typename Elem<kType>::T e[16];
  } out;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float f[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) f[v] = (static_cast<float>(acc[b][v]) * sx) * sw[4 * b + v];
    put4<kType>(out.w + b * (kWords / 4), f);
  }
  if (left >= 16) {
#pragma unroll
    for (int j = 0; j < kWords / 4; ++j) st16_any(y + j * (16 / sizeof(*y)), out.v[j]);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < left) y[e] = out.e[e];
  }
}

// 1 KB global -> LDS: lane l's 16 bytes at byte offset `off` to dst + 16 l.
__device__ __forceinline__ void copy_1k(__amdgpu_buffer_rsrc_t src, int8_t* dst, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void*)dst, 16, off, 0, 0, 0);
}

// Chunk order of a quad of rows (see below).
__device__ __forceinline__ int quad_key(int q) { return ((q << 1) & 3) ^ ((q >> 1) * 3); }

template <int BM, int BN, int WM, int WN, int kType>
__global__ __launch_bounds__(64 * WM * WN) void tile_kernel(LinearArgs g, int tiles_m, int tiles_n) {
  constexpr int kWaves = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles of a wave: tokens, channels
  constexpr int LX = BM / 16 / kWaves, LW = BN / 16 / kWaves;  // 1 KB loads of a wave a stage
  constexpr int kLoads = LX + LW;
  static_assert(TN % 4 == 0 && LX >= 1 && LW >= 1 && kWaves % 4 == 0, "tile shape");
  typedef typename Elem<kType>::T T;

  __shared__ __attribute__((aligned(1024))) int8_t s0[stage_bytes<BM, BN>()];
  __shared__ __attribute__((aligned(1024))) int8_t s1[stage_bytes<BM, BN>()];
  __shared__ __attribute__((aligned(1024))) int8_t s2[stage_bytes<BM, BN>()];
  __shared__ __attribute__((aligned(1024))) int8_t s3[stage_bytes<BM, BN>()];

  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // Workgroups go to the XCDs in turn; each XCD takes a run of tiles, ordered
  // in bands of 8 token tiles.
  const uint32_t total = static_cast<uint32_t>(tiles_m) * tiles_n;
  const uint32_t xcd = blockIdx.x % kXcds, local = blockIdx.x / kXcds;
  const uint32_t lin = xcd * (total / kXcds) + (xcd < total % kXcds ? xcd : total % kXcds) + local;
  const uint32_t band = 8 * static_cast<uint32_t>(tiles_n);
  const uint32_t b0 = lin / band * 8, in = lin % band;
  const uint32_t rows = static_cast<uint32_t>(tiles_m) - b0 < 8 ? static_cast<uint32_t>(tiles_m) - b0 : 8;
  const int64_t m0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(b0 + in % rows)) * BM;
  const int64_t n0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(in / rows)) * BN;

  const int nk = static_cast<int>(g.k / kBK);
  const int mrows = static_cast<int>(g.m - m0 < BM ? g.m - m0 : BM), nrows = static_cast<int>(g.n - n0 < BN ? g.n - n0 : BN);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + m0 * g.k, mrows * g.k);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.w + n0 * g.k, nrows * g.k);

  // Load l of a wave fills block l kWaves + wave: 16 rows of 64 bytes, lane l
  // the 16 bytes at row l / 4, place l % 4.
  const int lr = lane >> 2, lc = lane & 3;
  int xo[LX], wo[LW];
#pragma unroll
  for (int l = 0; l < LX; ++l) {
    const int row = 16 * (l * kWaves + wave) + lr;
    xo[l] = static_cast<int>((row < mrows ? row : mrows - 1) * g.k) + 16 * (lc ^ quad_key(lr >> 2));
  }
#pragma unroll
  for (int l = 0; l < LW; ++l) {
    const int row = 16 * (l * kWaves + wave) + lr;
    wo[l] = static_cast<int>((row < nrows ? row : nrows - 1) * g.k) + 16 * (lc ^ quad_key(wave & 3));
  }
  auto copy = [&](int8_t* stage, int kt) {
    const int q = (kt < nk ? kt : nk - 1) * kBK;
#pragma unroll
    for (int l = 0; l < LX; ++l)
      copy_1k(xr, stage + (l * kWaves + wave) * 1024, xo[l] + q);
#pragma unroll
    for (int l = 0; l < LW; ++l)
      copy_1k(wr, stage + BM * kBK + (l * kWaves + wave) * 1024, wo[l] + q);
  };
  const int xa = (wm * TM * 16 + i) * kBK + 16 * (h ^ quad_key(i >> 2));
  const int wa = BM * kBK + (wn * TN * 16 + 16 * (i >> 2) + (i & 3)) * kBK + 16 * (h ^ quad_key(i >> 2));
  u32x4 fx[2][TM], fw[2][TN];
  auto read = [&](const int8_t* stage, int set) {
#pragma unroll
    for (int t = 0; t < TN; ++t) fw[set][t] = ld16(stage + wa + (t >> 2) * (64 * kBK) + (t & 3) * (4 * kBK));
#pragma unroll
    for (int t = 0; t < TM; ++t) fx[set][t] = ld16(stage + xa + t * (16 * kBK));
  };
  i32x4 acc[TM][TN];
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
  auto multiply = [&](int set) {
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int b = 0; b < TN; ++b) acc[a][b] = mma8(fw[set][b], fx[set][a], acc[a][b]);
  };
  // Step kt: its fragments are in set; the next stage has to be whole, then
  // its fragments are read and this step's stage is filled again while the
  // matrix cores run.
  auto step = [&](int kt, int set, int8_t* mine, const int8_t* next) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this step's fragments have left the stage
    wait_vmcnt<(kStages - 2) * kLoads>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(next, set ^ 1);
    copy(mine, kt + kStages);
    multiply(set);
#pragma unroll
    for (int j = 0; j < TM + TN; ++j) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                        // LDS read
      if (j % 2 == 0 && j / 2 < kLoads) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);  // copy
      __builtin_amdgcn_sched_group_barrier(0x008, TM * TN / (TM + TN), 0);      // MFMA
    }
  };
  copy(s0, 0);
  copy(s1, 1);
  copy(s2, 2);
  copy(s3, 3);
  wait_vmcnt<(kStages - 1) * kLoads>();
  __builtin_amdgcn_s_barrier();
  read(s0, 0);
  int kt = 0;
  for (; kt + 4 <= nk; kt += 4) {
    step(kt, 0, s0, s1);
    step(kt + 1, 1, s1, s2);
    step(kt + 2, 0, s2, s3);
    step(kt + 3, 1, s3, s0);
  }
  if (kt < nk) step(kt, 0, s0, s1);
  if (kt + 1 < nk) step(kt + 1, 1, s1, s2);
  if (kt + 2 < nk) step(kt + 2, 0, s2, s3);
  wait_vmcnt<0>();  // no copy may be in flight when the workgroup's LDS is given on

  // Lane: tokens 16 a + i, channels 64 (b / 4) + 16 h + 4 (b % 4) + v: runs of
  // 16 neighbouring channels, 64 the four lanes of a token.
  T* y = static_cast<T*>(g.y);
#pragma unroll
  for (int c = 0; c < TN / 4; ++c) {
    const int64_t nc = n0 + wn * TN * 16 + 64 * c + 16 * h;
    float sw[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) sw[e] = g.sw[nc + e < g.n ? nc + e : g.n - 1];
#pragma unroll
    for (int a = 0; a < TM; ++a) {
      const int64_t m = m0 + wm * TM * 16 + 16 * a + i;
      if (m < g.m) store_run<kType>(y + m * g.n + nc, acc[a] + 4 * c, g.sx[m], sw, g.n - nc);
    }
  }
}

template <int BM, int BN, int WM, int WN>
hipError_t launch_tiles(const LinearArgs& g, int out_dtype, hipStream_t s) {
  const int tiles_m = static_cast<int>((g.m + BM - 1) / BM), tiles_n = static_cast<int>((g.n + BN - 1) / BN);
  auto kern = out_dtype == QLORA_F32   ? tile_kernel<BM, BN, WM, WN, QLORA_F32>
              : out_dtype == QLORA_F16 ? tile_kernel<BM, BN, WM, WN, QLORA_F16>
                                       : tile_kernel<BM, BN, WM, WN, QLORA_BF16>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles_m) * tiles_n), dim3(64 * WM * WN), 0, s, g, tiles_m, tiles_n);
  return hipGetLastError();
}

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
  if (m > 256) return launch_tiles<256, 256, 2, 4>(g, out_dtype, s);
  const int64_t tiles = ((m + kTM - 1) / kTM) * ((n + kTN - 1) / kTN);
  auto kern = out_dtype == QLORA_F32   ? linear_kernel<QLORA_F32>
              : out_dtype == QLORA_F16 ? linear_kernel<QLORA_F16>
                                       : linear_kernel<QLORA_BF16>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace qlora
