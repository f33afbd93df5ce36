// The 8-bit product Y = (X W^T) with one scale a token and one a channel.
//
// Codes are contracted with v_mfma_i32_16x16x64_i8 into exact 32-bit integer
// sums (k 128^2 < 2^31), so the sums do not depend on the order or the split
// of the work; the scales enter once, at the end.
//
// What bounds it, by size (MI355X; graph replays, bf16 out):
//   - Few tokens: the weight's bytes. 1 x 4096 x 4096 (m x n x k) 5.5 us, 16 x
//     11008 x 4096 10.8 us (45 MB; a large copy moves 4.7 TB/s here, read and
//     written).
//   - Hundreds of tokens: the copies into LDS. 333 x 5003 x 4160 takes 17.6 us in
//     64 x 128 tiles, 16.5 us with reads and products left out, 6.0 us with the
//     copies left out too: 190 MB out of the L2 caches at 18 TB/s (20-21 is the
//     most that any tile reached, 85-90 bytes/ns a CU). A deeper ring or two
//     groups of waves on that tile gain nothing.
//   - Thousands: the matrix cores and their power. 4096 x 8192 x 8192 206 us
//     (2670 TOP/s); the matrix cores are busy 68% of the cycles, at 1.8 GHz. With
//     v_mfma_i32_32x32x32_i8 in 128 x 128 tiles a wave (a third fewer LDS reads)
//     the cycles are as many, at 1.64 GHz: 236 us.
#include "bufmem.h"
#include "elem.h"
#include "int8_tiles.h"

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
  int64_t ldy;  // a row of y; n but for a part of the channels
};

// ---------------------------------------------------------------------------
// Tiles through LDS: both operands are copied from memory into a ring of units
// (128 codes of the tile's rows), read as fragments and multiplied. 128 codes
// are a cache line of a row: copies of 64-code rows moved half as many codes a
// cycle (4096 x 22016 x 8192: 632 us, 603 us with whole lines).
// ---------------------------------------------------------------------------
constexpr int kUnit = 128;
constexpr int kXcds = 8;
constexpr int kNowhere = 0x70000000;  // an offset past every tile's range, also with one of a tile added

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
// of one more, so that half of the codes have a unit's time more to arrive: the
// 256 x 256 tile's five parts are all of LDS (4096 x 8192 x 8192: 212 us with
// four, 206 with five).
// KS: groups of WM x WN waves that share the contraction of one tile, each with
// a ring of its own; their sums are added through LDS at the end. For tiles so
// small that one group keeps too few copies in flight (128 x 4096 x 4096 in 32
// x 64 tiles: 8.6 us with two groups).
template <int BM, int BN, int WM, int WN, int KS, int P, int kType>
__global__ __launch_bounds__(64 * WM * WN * KS) void tile_kernel(LinearArgs g, int tiles_m, int tiles_n) {
  constexpr int kWaves = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles of a wave: tokens, channels
  constexpr int LX = BM / 8 / kWaves, LW = BN / 8 / kWaves;  // 1 KB copies of a wave a part
  constexpr int kLoads = LX + LW;
  constexpr int S = P / 2;        // units that the ring holds whole
  constexpr bool kOdd = P % 2 != 0;
  constexpr int kTurn = kOdd ? P : S;  // units after which parts lie in the same places again
  static_assert(TN % 4 == 0 && BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "tile shape");
  static_assert(P >= 4 && P <= 8 && (!kOdd || BM == BN), "ring");
  // groups whose sums fit the channels' part of the ring
  constexpr int kFit = KS * kUnit / (4 * BM);
  static_assert(KS == 1 || (kFit >= 1 && (KS - 1 + kFit - 1) / kFit <= P / 2), "sums of the groups");
  typedef typename Elem<kType>::T T;

  // one array a part: the compiler can then tell a copy into one part from the
  // reads of another, and waits for none of them by itself
  __shared__ __attribute__((aligned(1024))) int8_t p0[KS * BM * kUnit];
  __shared__ __attribute__((aligned(1024))) int8_t p1[KS * BN * kUnit];
  __shared__ __attribute__((aligned(1024))) int8_t p2[KS * BM * kUnit];
  __shared__ __attribute__((aligned(1024))) int8_t p3[KS * BN * kUnit];
  __shared__ __attribute__((aligned(1024))) int8_t p4[P > 4 ? KS * BM * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) int8_t p5[P > 5 ? KS * BN * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) int8_t p6[P > 6 ? KS * BM * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) int8_t p7[P > 7 ? KS * BN * kUnit : 16];
  int8_t* const ring[8] = {p0, p1, p2, p3, p4, p5, p6, p7};

  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, h = lane >> 4;
  const int wave_all = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = wave_all / kWaves, wave = wave_all % kWaves;
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

  // This group's units [u0, u0 + turns): the same number for all groups, the
  // last ones' past the end of the contraction.
  const int units = static_cast<int>((g.k + kUnit - 1) / kUnit);
  const int turns = (units + KS - 1) / KS, u0 = group * turns;
  const int mrows = static_cast<int>(g.m - m0 < BM ? g.m - m0 : BM), nrows = static_cast<int>(g.n - n0 < BN ? g.n - n0 : BN);
  // Ranges of the tile's own rows: what is read at an offset past them is zero.
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + m0 * g.k, mrows * g.k);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.w + n0 * g.k, nrows * g.k);

  // Copy l of a wave fills block l kWaves + wave of a part: 8 rows of 128
  // bytes, lane l the 16 bytes at row l / 8, place l % 8. A row's chunk c
  // stands at place c ^ key(row). The 16 lanes that read one chunk column
  // then fall on 16 different 16-byte columns of the banks, both as 16
  // neighbouring lanes and as four quads of lanes out of two columns.
  // Rows past the tile's last lie past its range.
  const int lr = lane >> 3, lc = lane & 7;
  const int k32 = static_cast<int>(g.k);
  int xc[LX], wo[LW];  // byte in the row's unit; offset without rows of blocks
#pragma unroll
  for (int l = 0; l < LX; ++l) xc[l] = 16 * (lc ^ ((lr >> 1) + 4 * ((l * kWaves + wave) & 1)));
#pragma unroll
  for (int l = 0; l < LW; ++l)
    wo[l] = (8 * wave + lr) * k32 + 16 * (lc ^ (2 * (((l * kWaves + wave) >> 1) & 3) + ((lr >> 1) & 1)));
  const int xrow = (8 * wave + lr) * k32;
  // Codes behind the contraction's end (in the second half of its last unit,
  // and in units past it) become zeros on the tokens' side, so their products
  // vanish whatever the channels' side holds.
  auto copy_x = [&](int8_t* to, int u) {
    const int q = (u0 + u) * kUnit;
#pragma unroll
    for (int l = 0; l < LX; ++l) {
      const int at = xc[l] < k32 - q ? xrow + xc[l] : kNowhere;
      copy_1k(xr, to + (group * BM / 8 + l * kWaves + wave) * 1024, at + (8 * l * kWaves * k32 + q));
    }
  };
  auto copy_w = [&](int8_t* to, int u) {
    const int q = (u0 + u < units ? u0 + u : units - 1) * kUnit;
#pragma unroll
    for (int l = 0; l < LW; ++l)
      copy_1k(wr, to + (group * BN / 8 + l * kWaves + wave) * 1024, wo[l] + (8 * l * kWaves * k32 + q));
  };
  // Fragments of a unit's first or second 64 codes. Token tile t reads rows
  // 16 t + i; channel tile t rows 64 (t / 4) + 16 (i / 4) + 4 (t % 4) + i % 4,
  // which leaves a lane with runs of 16 neighbouring channels. Both keys are
  // i / 2.
  const int xa = (group * BM + wm * TM * 16 + i) * kUnit;
  const int wa = (group * BN + wn * TN * 16 + 16 * (i >> 2) + (i & 3)) * kUnit;
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
  // Lane: tokens 16 a + i, channels 64 (b / 4) + 16 h + 4 (b % 4) + v: runs of
  // 16 neighbouring channels, 64 the four lanes of a token. Tiles that leave
  // registers for their scales load these in front of the contraction.
  constexpr bool kEarly = TM * TN <= 16;
  float sx[TM], sw[kEarly ? TN / 4 : 1][16];
  auto load_scales = [&](int c) {
    const int64_t nc = n0 + wn * TN * 16 + 64 * c + 16 * h;
#pragma unroll
    for (int e = 0; e < 16; ++e) sw[kEarly ? c : 0][e] = g.sw[nc + e < g.n ? nc + e : g.n - 1];
    if (c > 0) return;
#pragma unroll
    for (int a = 0; a < TM; ++a) {
      const int64_t m = m0 + wm * TM * 16 + 16 * a + i;
      sx[a] = g.sx[m < g.m ? m : g.m - 1];
    }
  };
  if (kEarly) {
#pragma unroll
    for (int c = 0; c < TN / 4; ++c) load_scales(c);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p % 2 == 0) copy_x(ring[p], p / 2);
    else copy_w(ring[p], p / 2);
  }
  wait_vmcnt<(S - 1) * kLoads + (kOdd ? LX : 0)>();
  __builtin_amdgcn_s_barrier();
  read(p0, p1, 0);
  int u = 0;
  for (; u + kTurn <= turns; u += kTurn) {
#pragma unroll
    for (int j = 0; j < kTurn; ++j)
      unit(u + j, ring[2 * j % P], ring[(2 * j + 1) % P], ring[(2 * j + 2) % P], ring[(2 * j + 3) % P]);
  }
#pragma unroll
  for (int j = 0; j < kTurn - 1; ++j)
    if (u + j < turns)
      unit(u + j, ring[2 * j % P], ring[(2 * j + 1) % P], ring[(2 * j + 2) % P], ring[(2 * j + 3) % P]);
  wait_vmcnt<0>();  // no copy may be in flight when the ring is used again, here or by the next workgroup

  if (KS > 1) {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __syncthreads();  // every group's copies and reads have ended
    auto sums = [&](int gr) {  // group gr's
      int8_t* at = ring[1 + 2 * ((gr - 1) / (kFit > 0 ? kFit : 1))] + (gr - 1) % (kFit > 0 ? kFit : 1) * (BM * BN * 4);
      return reinterpret_cast<i32x4*>(at) + wave * (TM * TN * 64) + lane;
    };
#pragma unroll
    for (int gr = 1; gr < KS; ++gr) {
      if (group != gr) continue;
      i32x4* to = sums(gr);
#pragma unroll
      for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b) to[(a * TN + b) * 64] = acc[a][b];
    }
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int gr = 1; gr < KS; ++gr) {
      const i32x4* from = sums(gr);
#pragma unroll
      for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b) acc[a][b] += from[(a * TN + b) * 64];
    }
  }

  T* y = static_cast<T*>(g.y);
#pragma unroll
  for (int c = 0; c < TN / 4; ++c) {
    const int64_t nc = n0 + wn * TN * 16 + 64 * c + 16 * h;
    if (!kEarly) load_scales(c);
#pragma unroll
    for (int a = 0; a < TM; ++a) {
      const int64_t m = m0 + wm * TM * 16 + 16 * a + i;
      if (m < g.m) store_run<kType>(y + m * g.ldy + nc, acc[a] + 4 * c, sx[a], sw[kEarly ? c : 0], g.n - nc);
    }
  }
}

template <int I>
hipError_t launch_tiles(const LinearArgs& g, int out_dtype, hipStream_t s) {
  constexpr Shape t = kShapes[I];
  constexpr int BM = t.bm, BN = t.bn, WM = t.wm, WN = t.wn, KS = t.groups, P = t.parts;
  const int tiles_m = static_cast<int>((g.m + BM - 1) / BM), tiles_n = static_cast<int>((g.n + BN - 1) / BN);
  auto kern = out_dtype == QLORA_F32   ? tile_kernel<BM, BN, WM, WN, KS, P, QLORA_F32>
              : out_dtype == QLORA_F16 ? tile_kernel<BM, BN, WM, WN, KS, P, QLORA_F16>
                                       : tile_kernel<BM, BN, WM, WN, KS, P, QLORA_BF16>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles_m) * tiles_n), dim3(t.threads()), 0, s, g, tiles_m, tiles_n);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// At most 16 tokens and few channels: the weight is streamed once, bound by
// memory. A workgroup takes 16 channels (so 4096 channels fill the 256 CUs);
// its waves split the contraction, read their runs of the 16 rows straight
// into registers, and add their integer sums through LDS.
// One token, 4096 x 4096: 5.5 us (graph replays; 4.8 TB/s behind a launch's
// 2 us); 4 to 16 waves and 2 to 8 loads in flight measure alike. The 16 x 64 and
// 32 x 64 tiles above read the tokens once for 64 channels, not for 16, and cost
// more to start. Both, us, here / there:
//   channels              1024      2048       4096       5120       6144       8128
//   k 4096,  1 token     4.4/6.2   4.7/6.3    5.5/6.5    7.5/6.5    7.5/6.8    8.1/7.8
//   k 4096,  16 tokens   5.7/6.3   6.0/6.6    6.2/6.7    9.6/6.8    9.6/7.0    9.7/8.1
//   k 11008, 1 token     8.8/11.7  8.9/11.7  10.6/18.0  20.0/19.4  20.8/21.0  22.0/22.6
//   k 11008, 16 tokens  12.7/12.4 12.8/12.7  14.1/19.9  26.3/21.8  27.5/23.6  29.3/25.1
// Up to 4096 channels, one round of workgroups, this kernel is the faster one.
// From there to the bound at 8191 the tiles mostly are, by up to 30% at 16
// tokens: the bound stands above the crossing and is no part of the tiles' cost.
// ---------------------------------------------------------------------------
constexpr int kDecodeWaves = 8;
constexpr int kDecodeSteps = 4;  // 64-code steps of a wave a pass

template <int kType>
__global__ __launch_bounds__(64 * kDecodeWaves) void decode_kernel(LinearArgs g) {
  __shared__ int part[kDecodeWaves][256];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int steps = static_cast<int>(g.k / 64);
  const int8_t* wp = g.w + (n0 + i < g.n ? n0 + i : g.n - 1) * g.k + 16 * h;
  const int8_t* xp = g.x + (i < g.m ? i : g.m - 1) * g.k + 16 * h;
  i32x4 acc = {0, 0, 0, 0};
  for (int base = 0; base < steps; base += kDecodeWaves * kDecodeSteps) {
    // this wave's steps of the pass; past the end the last one is read again
    // and multiplied by zeros
    const int s0 = base + wave * kDecodeSteps;
    u32x4 wf[kDecodeSteps], xf[kDecodeSteps];
#pragma unroll
    for (int j = 0; j < kDecodeSteps; ++j) {
      const int q = 64 * (s0 + j < steps ? s0 + j : steps - 1);
      wf[j] = ld16(wp + q);
      xf[j] = ld16(xp + q);
    }
#pragma unroll
    for (int j = 0; j < kDecodeSteps; ++j) {
      if (s0 + j >= steps) xf[j] = u32x4{0, 0, 0, 0};
      acc = mma8(wf[j], xf[j], acc);
    }
  }
  *reinterpret_cast<i32x4*>(&part[wave][4 * lane]) = acc;
  __syncthreads();
  // output tid: token tid / 16, channel tid % 16
  const int tok = tid >> 4, ch = tid & 15;
  if (tid >= 256 || tok >= g.m || n0 + ch >= g.n) return;
  const int at = 4 * (tok + 16 * (ch >> 2)) + (ch & 3);
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kDecodeWaves; ++w) sum += part[w][at];
  static_cast<typename Elem<kType>::T*>(g.y)[tok * g.ldy + n0 + ch] =
      Elem<kType>::put((static_cast<float>(sum) * g.sx[tok]) * g.sw[n0 + ch]);
}

hipError_t launch_decode(const LinearArgs& g, int out_dtype, hipStream_t s) {
  auto kern = out_dtype == QLORA_F32   ? decode_kernel<QLORA_F32>
              : out_dtype == QLORA_F16 ? decode_kernel<QLORA_F16>
                                       : decode_kernel<QLORA_BF16>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((g.n + 15) / 16)), dim3(64 * kDecodeWaves), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_shape(int shape, const LinearArgs& g, int out_dtype, hipStream_t s) {
  switch (shape) {
    case 0:
      return launch_tiles<0>(g, out_dtype, s);
    case 1:
      return launch_tiles<1>(g, out_dtype, s);
    case 2:
      return launch_tiles<2>(g, out_dtype, s);
    case 3:
      return launch_tiles<3>(g, out_dtype, s);
    case 4:
      return launch_tiles<4>(g, out_dtype, s);
    case 5:
      return launch_tiles<5>(g, out_dtype, s);
    case 6:
      return launch_tiles<6>(g, out_dtype, s);
  }
  return hipErrorInvalidValue;  // int8_linear_fits refuses these sizes
}

}  // namespace

bool int8_linear_fits(int64_t m, int64_t n, int64_t k) { return decodes(m, n) || pick_shape(m, n, k).shape >= 0; }

hipError_t launch_int8_linear(const int8_t* w, const float* w_scale, int64_t n, int64_t k, const int8_t* x,
                              const float* x_scale, int64_t m, int out_dtype, void* y, hipStream_t s) {
  LinearArgs g{w, w_scale, x, x_scale, y, m, n, k, n};
  if (decodes(m, n)) return launch_decode(g, out_dtype, s);
  const Pick one = pick_shape(m, n, k);
  const int64_t cols = full_rounds(m, n, k, one);
  if (cols > 0) {
    g.n = cols;
    const hipError_t e = launch_shape(0, g, out_dtype, s);
    if (e != hipSuccess) return e;
    g.w = w + cols * k;
    g.sw = w_scale + cols;
    g.y = static_cast<char*>(y) + cols * (out_dtype == QLORA_F32 ? 4 : 2);
    g.n = n - cols;
    return launch_shape(pick_shape(m, g.n, k).shape, g, out_dtype, s);
  }
  return launch_shape(one.shape, g, out_dtype, s);
}

}  // namespace qlora
