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
constexpr int kUnit = 128;  // contraction codes of a stage: a whole cache line of a row
constexpr int kXcds = 8;

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

// P: parts of the LDS ring. A unit of 128 codes is two parts, the tokens' and
// the channels'; the ring holds P / 2 units, and with an odd P the tokens' part
// of one more, so that half of the codes have a unit's time more to arrive.
template <int BM, int BN, int WM, int WN, int P, int kType>
__global__ __launch_bounds__(64 * WM * WN) void tile_kernel(LinearArgs g, int tiles_m, int tiles_n) {
  constexpr int kWaves = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles of a wave: tokens, channels
  constexpr int LX = BM / 8 / kWaves, LW = BN / 8 / kWaves;  // 1 KB copies of a wave a stage
  constexpr int kLoads = LX + LW;
  constexpr int S = P / 2;        // units that the ring holds whole
  constexpr bool kOdd = P % 2 != 0;
  constexpr int kTurn = kOdd ? P : S;  // units after which parts lie in the same places again
  static_assert(TN % 4 == 0 && BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "tile shape");
  static_assert(P >= 4 && P <= 8 && (!kOdd || BM == BN), "ring");
  typedef typename Elem<kType>::T T;

  // one array a part: the compiler can then tell a copy into one part from the
  // reads of another, and waits for none of them by itself
  __shared__ __attribute__((aligned(1024))) int8_t p0[BM * kUnit];
  __shared__ __attribute__((aligned(1024))) int8_t p1[BN * kUnit];
  __shared__ __attribute__((aligned(1024))) int8_t p2[BM * kUnit];
  __shared__ __attribute__((aligned(1024))) int8_t p3[BN * kUnit];
  __shared__ __attribute__((aligned(1024))) int8_t p4[P > 4 ? BM * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) int8_t p5[P > 5 ? BN * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) int8_t p6[P > 6 ? BM * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) int8_t p7[P > 7 ? BN * kUnit : 16];
  int8_t* const ring[8] = {p0, p1, p2, p3, p4, p5, p6, p7};

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

  const int units = static_cast<int>((g.k + kUnit - 1) / kUnit), whole = static_cast<int>(g.k / kUnit);
  const int mrows = static_cast<int>(g.m - m0 < BM ? g.m - m0 : BM), nrows = static_cast<int>(g.n - n0 < BN ? g.n - n0 : BN);
  // Ranges of the tile's own rows: the last unit of a contraction that is no
  // multiple of 128 reads past its rows, into the next row or, past the last
  // one, into zeros; neither is multiplied.
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + m0 * g.k, mrows * g.k);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.w + n0 * g.k, nrows * g.k);

  // Copy l of a wave fills block l kWaves + wave of a stage: 8 rows of 128
  // bytes, lane l the 16 bytes at row l / 8, place l % 8. A row's chunk c
  // stands at place c ^ key(row). The 16 lanes that read one chunk column
  // then fall on 16 different 16-byte columns of the banks, both as 16
  // neighbouring lanes and as four quads of lanes out of two columns.
  const int lr = lane >> 3, lc = lane & 7;
  int xo[LX], wo[LW];
#pragma unroll
  for (int l = 0; l < LX; ++l) {
    const int row = 8 * (l * kWaves + wave) + lr;
    xo[l] = static_cast<int>((row < mrows ? row : mrows - 1) * g.k) + 16 * (lc ^ ((row >> 1) & 7));
  }
#pragma unroll
  for (int l = 0; l < LW; ++l) {
    const int row = 8 * (l * kWaves + wave) + lr;
    wo[l] = static_cast<int>((row < nrows ? row : nrows - 1) * g.k) +
            16 * (lc ^ (2 * ((row >> 4) & 3) + ((row >> 1) & 1)));
  }
  auto copy_x = [&](int8_t* to, int u) {
    const int q = (u < units ? u : units - 1) * kUnit;
#pragma unroll
    for (int l = 0; l < LX; ++l) copy_1k(xr, to + (l * kWaves + wave) * 1024, xo[l] + q);
  };
  auto copy_w = [&](int8_t* to, int u) {
    const int q = (u < units ? u : units - 1) * kUnit;
#pragma unroll
    for (int l = 0; l < LW; ++l) copy_1k(wr, to + (l * kWaves + wave) * 1024, wo[l] + q);
  };
  // Fragments of the stage's first or second 64 codes. Token tile t reads rows
  // 16 t + i; channel tile t rows 64 (t / 4) + 16 (i / 4) + 4 (t % 4) + i % 4,
  // which leaves a lane with runs of 16 neighbouring channels. Both keys are
  // i / 2.
  const int xa = (wm * TM * 16 + i) * kUnit;
  const int wa = (wn * TN * 16 + 16 * (i >> 2) + (i & 3)) * kUnit;
  const int place[2] = {16 * (h ^ (i >> 1)), 16 * ((4 + h) ^ (i >> 1))};
  u32x4 fx[2][TM], fw[2][TN];
  auto read = [&](const int8_t* x, const int8_t* w, int half) {
#pragma unroll
    for (int t = 0; t < TN; ++t)
      fw[half][t] = ld16(w + wa + place[half] + (t >> 2) * (64 * kUnit) + (t & 3) * (4 * kUnit));
#pragma unroll
    for (int t = 0; t < TM; ++t) fx[half][t] = ld16(x + xa + place[half] + t * (16 * kUnit));
  };
  i32x4 acc[TM][TN];
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
  auto multiply = [&](int half) {
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int b = 0; b < TN; ++b) acc[a][b] = mma8(fw[half][b], fx[half][a], acc[a][b]);
  };
  // Unit u, whose first half's fragments are in registers: its second half is
  // read while the first is multiplied; then the next unit has to be whole,
  // its first half is read and this unit's parts filled again while the second
  // is multiplied. One barrier a unit.
  auto unit = [&](int u, int8_t* x, int8_t* w, const int8_t* next_x, const int8_t* next_w) {
    read(x, w, 1);
    multiply(0);
#pragma unroll
    for (int j = 0; j < TM + TN; ++j) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                    // LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, TM * TN / (TM + TN), 0);  // MFMA
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the fragments have left this unit's parts
    wait_vmcnt<(S - 2) * kLoads + (kOdd ? LX : 0)>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (kOdd) {
      copy_w(x, u + S);
      copy_x(w, u + S + 1);
    } else {
      copy_x(x, u + S);
      copy_w(w, u + S);
    }
    read(next_x, next_w, 0);
    multiply(1);
#pragma unroll
    for (int j = 0; j < TM + TN; ++j) {
      if (j < kLoads) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);  // copy
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, TM * TN / (TM + TN), 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p % 2 == 0) copy_x(ring[p], p / 2);
    else copy_w(ring[p], p / 2);
  }
  wait_vmcnt<(S - 1) * kLoads + (kOdd ? LX : 0)>();
  __builtin_amdgcn_s_barrier();
  read(p0, p1, 0);
  int u = 0;
  for (; u + kTurn <= whole; u += kTurn) {
#pragma unroll
    for (int j = 0; j < kTurn; ++j)
      unit(u + j, ring[2 * j % P], ring[(2 * j + 1) % P], ring[(2 * j + 2) % P], ring[(2 * j + 3) % P]);
  }
#pragma unroll
  for (int j = 0; j < kTurn - 1; ++j)
    if (u + j < whole)
      unit(u + j, ring[2 * j % P], ring[(2 * j + 1) % P], ring[(2 * j + 2) % P], ring[(2 * j + 3) % P]);
  if (whole < units) multiply(0);
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

template <int BM, int BN, int WM, int WN, int P>
hipError_t launch_tiles(const LinearArgs& g, int out_dtype, hipStream_t s) {
  const int tiles_m = static_cast<int>((g.m + BM - 1) / BM), tiles_n = static_cast<int>((g.n + BN - 1) / BN);
  auto kern = out_dtype == QLORA_F32   ? tile_kernel<BM, BN, WM, WN, P, QLORA_F32>
              : out_dtype == QLORA_F16 ? tile_kernel<BM, BN, WM, WN, P, QLORA_F16>
                                       : tile_kernel<BM, BN, WM, WN, P, QLORA_BF16>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles_m) * tiles_n), dim3(64 * WM * WN), 0, s, g, tiles_m, tiles_n);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Few tokens: the weight is streamed once, bound by memory. A workgroup of 16
// waves takes 16 channels; its waves split the contraction, each reading its
// runs of the 16 rows straight into registers, all loads in flight at once,
// and add their integer sums through LDS.
// ---------------------------------------------------------------------------
constexpr int kDecodeWaves = 8;
constexpr int kDecodeBlocks = 256;

// J: 64-code steps of a wave a pass; TT: tiles of 16 tokens. kOne: one pass
// covers the contraction, so the tokens stay in registers while the workgroup
// goes through its channels, and the next weight rows are on their way while
// the sums of the last ones are added.
template <int J, int TT, bool kOne, int kType>
__global__ __launch_bounds__(64 * kDecodeWaves) void decode_kernel(LinearArgs g, int groups) {
  __shared__ int part[2][kDecodeWaves][TT * 256];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int steps = static_cast<int>(g.k / 64);
  const int8_t* xp[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) xp[t] = g.x + (16 * t + i < g.m ? 16 * t + i : g.m - 1) * g.k + 16 * h;
  // Step j of this wave in the pass at `base`; past the end the last step is
  // read again and multiplied by zeros.
  auto at = [&](int base, int j) {
    const int s = base + wave * J + j;
    return 64 * (s < steps ? s : steps - 1);
  };
  u32x4 wf[J], xf[TT][J];
  auto read_w = [&](int group, int base) {
    const int64_t n = static_cast<int64_t>(group) * 16 + i;
    const int8_t* wp = g.w + (n < g.n ? n : g.n - 1) * g.k + 16 * h;
#pragma unroll
    for (int j = 0; j < J; ++j) wf[j] = ld16(wp + at(base, j));
  };
  auto read_x = [&](int base) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        xf[t][j] = ld16(xp[t] + at(base, j));
        if (base + wave * J + j >= steps) xf[t][j] = u32x4{0, 0, 0, 0};
      }
  };
  read_w(blockIdx.x, 0);
  read_x(0);
  int turn = 0;
  for (int group = blockIdx.x; group < groups; group += gridDim.x, turn ^= 1) {
    i32x4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    auto multiply = [&] {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = mma8(wf[j], xf[t][j], acc[t]);
    };
    if (kOne) {
      multiply();
      const int next = group + gridDim.x;
      if (next < groups) read_w(next, 0);
    } else {
      for (int base = 0; base < steps; base += kDecodeWaves * J) {
        if (base > 0 || group != static_cast<int>(blockIdx.x)) {
          read_w(group, base);
          read_x(base);
        }
        multiply();
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) *reinterpret_cast<i32x4*>(&part[turn][wave][t * 256 + 4 * lane]) = acc[t];
    __syncthreads();  // the other turn's sums have been read by all in front of this
    // output e: token e / 16, channel e % 16
    const int64_t n = static_cast<int64_t>(group) * 16 + (tid & 15);
#pragma unroll
    for (int e = tid; e < TT * 256; e += 64 * kDecodeWaves) {
      const int64_t m = e >> 4;
      if (m >= g.m || n >= g.n) continue;
      const int from = (e >> 8) * 256 + 4 * (((e >> 4) & 15) + 16 * ((e & 15) >> 2)) + (e & 3);
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kDecodeWaves; ++w) sum += part[turn][w][from];
      static_cast<typename Elem<kType>::T*>(g.y)[m * g.n + n] =
          Elem<kType>::put((static_cast<float>(sum) * g.sx[m]) * g.sw[n]);
    }
  }
}

template <int J, int TT, bool kOne>
hipError_t launch_decode(const LinearArgs& g, int out_dtype, hipStream_t s) {
  const int groups = static_cast<int>((g.n + 15) / 16);
  const int blocks = kOne && groups > kDecodeBlocks ? kDecodeBlocks : groups;
  auto kern = out_dtype == QLORA_F32   ? decode_kernel<J, TT, kOne, QLORA_F32>
              : out_dtype == QLORA_F16 ? decode_kernel<J, TT, kOne, QLORA_F16>
                                       : decode_kernel<J, TT, kOne, QLORA_BF16>;
  hipLaunchKernelGGL(kern, dim3(blocks), dim3(64 * kDecodeWaves), 0, s, g, groups);
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
  if (m <= 16) {
    if (k <= 2048) return launch_decode<4, 1, true>(g, out_dtype, s);
    if (k <= 4096) return launch_decode<8, 1, true>(g, out_dtype, s);
    return launch_decode<4, 1, false>(g, out_dtype, s);
  }
  if (m <= 32) {
    if (k <= 2048) return launch_decode<4, 2, true>(g, out_dtype, s);
    if (k <= 4096) return launch_decode<8, 2, true>(g, out_dtype, s);
    return launch_decode<4, 2, false>(g, out_dtype, s);
  }
  if (m > 32) return launch_tiles<256, 256, 2, 4, 5>(g, out_dtype, s);
  const int64_t tiles = ((m + kTM - 1) / kTM) * ((n + kTN - 1) / kTN);
  auto kern = out_dtype == QLORA_F32   ? linear_kernel<QLORA_F32>
              : out_dtype == QLORA_F16 ? linear_kernel<QLORA_F16>
                                       : linear_kernel<QLORA_BF16>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, g);
  return hipGetLastError();
}

}  // namespace qlora
