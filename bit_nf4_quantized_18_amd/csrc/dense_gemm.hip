// The matrix product of a weight that was restored to 16 bits in the workspace:
//   forward of a gated block: [G | U] = X W16^T + the adapters, P = act(G) U
//   backward data:            dX = dY W16 + dH A, from the restored transpose
//
// The fused kernels of gemm_kernels.hip restore a weight anew for every 256 tokens,
// and what they restore sets the pace of their steps. From a few hundred tokens on
// it is cheaper to restore the weight once (2.5 bytes of memory a weight) and to
// multiply it as it is.
//
// Rows of bytes as in the 8-bit product: both operands are copied from memory into
// a ring of units (128 bytes of the tile's rows, 64 elements), read as fragments
// half a unit ahead and multiplied by v_mfma_f32_16x16x32. The adapter's slots
// follow as more contraction, with operands straight from memory and H or dH in three
// 16-bit terms (0.6% of this call at rank 16, 9% at 64). 2048 x 22016 x 4096, gated: 275 to 300
// us (1.23 to 1.34 PFLOP/s; the library's 8192^3 product reaches 1.52) behind 44 to 48 us
// of restoring (5.8 TB/s); the fused product takes 396 in all.
#include "bufmem.h"
#include "dense_rule.h"
#include "gate.h"
#include "internal.h"
#include "lora_transpose.h"
#include "mfma.h"
#include "nf4_lut.h"

namespace qlora {
namespace {

struct DenseArgs {
  const uint8_t* w;  // n rows (gated: 2 n, gate's above up's) of kb bytes
  const uint8_t* x;  // m rows of kb bytes
  int64_t m, n, kb;
  int64_t up;         // gated: weight rows from an output's gate row to its up row
  const uint16_t* ha;  // m x 3 rpad: the adapter's slots as terms (put_terms, mfma.h)
  const uint16_t* hb;  // their rows of a channel: hb_lim slots at hb_ld, up's after `shift` others
  int64_t hb_ld;
  int hb_lim, rpad, shift;
  uint16_t* y;  // m x n at ldy; gated: [G | U] at ldy = 2 up, may be null
  int64_t ldy;
  uint16_t* p;  // gated: m x up
  int act;
};

constexpr int kUnit = 128;  // bytes of a row
constexpr int kXcds = 8;
constexpr int kNowhere = 0x70000000;  // an offset past every tile's range, also with one of a tile added

// 1 KB global -> LDS: lane l's 16 bytes at byte offset `off` to dst + 16 l.
__device__ __forceinline__ void copy_1k(__amdgpu_buffer_rsrc_t src, uint8_t* dst, int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void*)dst, 16, off, 0, 0, 0);
}

// BM x BN tiles, KS groups of WM x WN waves that share the contraction, P parts of
// a group's ring: a unit is two parts, the tokens' and the channels', and with an
// odd P the tokens' part of one more unit has its place too.
// kGated: BN weight rows are BN / 2 outputs; blocks of eight rows of the channels'
// part are gate's and up's in turn.
template <int BM, int BN, int WM, int WN, int KS, int P, bool kF16, bool kGated>
__global__ __launch_bounds__(64 * WM * WN * KS) void dense_kernel(DenseArgs g, int tiles_m, int tiles_n) {
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

  // one array a part: the compiler can then tell a copy into one part from the
  // reads of another, and waits for none of them by itself
  __shared__ __attribute__((aligned(1024))) uint8_t p0[KS * BM * kUnit];
  __shared__ __attribute__((aligned(1024))) uint8_t p1[KS * BN * kUnit];
  __shared__ __attribute__((aligned(1024))) uint8_t p2[KS * BM * kUnit];
  __shared__ __attribute__((aligned(1024))) uint8_t p3[KS * BN * kUnit];
  __shared__ __attribute__((aligned(1024))) uint8_t p4[P > 4 ? KS * BM * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t p5[P > 5 ? KS * BN * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t p6[P > 6 ? KS * BM * kUnit : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t p7[P > 7 ? KS * BN * kUnit : 16];
  uint8_t* const ring[8] = {p0, p1, p2, p3, p4, p5, p6, p7};

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
  constexpr int BO = kGated ? BN / 2 : BN;  // outputs of a tile
  const int64_t n0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(in / rows)) * BO;

  // This group's units [u0, u0 + turns): the same number for all groups, the
  // last ones' past the end of the contraction.
  const int units = static_cast<int>((g.kb + kUnit - 1) / kUnit);
  const int turns = (units + KS - 1) / KS, u0 = group * turns;
  const int mrows = static_cast<int>(g.m - m0 < BM ? g.m - m0 : BM), nrows = static_cast<int>(g.n - n0 < BO ? g.n - n0 : BO);
  // Ranges of the tile's own rows: what is read at an offset past them is zero.
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + m0 * g.kb, mrows * g.kb);
  // Gated: the odd blocks of eight rows are up's. Where the waves are even in
  // number a wave copies blocks of one parity alone.
  constexpr bool kEven = kWaves % 2 == 0;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.w + (n0 + (kGated && kEven && (wave & 1) ? g.up : 0)) * g.kb, nrows * g.kb);
  const __amdgpu_buffer_rsrc_t ur = make_rsrc(g.w + (n0 + (kGated && !kEven ? g.up : 0)) * g.kb, nrows * g.kb);

  // Copy l of a wave fills block l kWaves + wave of a part: 8 rows of 128
  // bytes, lane l the 16 bytes at row l / 8, place l % 8. A row's chunk c
  // stands at place c ^ key(row). The 16 lanes that read one chunk column
  // then fall on 16 different 16-byte columns of the banks, both as 16
  // neighbouring lanes and as four quads of lanes out of two columns.
  // Rows past the tile's last lie past its range.
  const int lr = lane >> 3, lc = lane & 7;
  const int k32 = static_cast<int>(g.kb);
  int xc[LX], wc[LW], wo[LW];  // byte in the row's unit; offset without rows of blocks
#pragma unroll
  for (int l = 0; l < LX; ++l) xc[l] = 16 * (lc ^ ((lr >> 1) + 4 * ((l * kWaves + wave) & 1)));
#pragma unroll
  for (int l = 0; l < LW; ++l) {
    wc[l] = 16 * (lc ^ (2 * (((l * kWaves + wave) >> 1) & 3) + ((lr >> 1) & 1)));
    wo[l] = ((kGated ? 8 * (wave >> 1) : 8 * wave) + lr) * k32 + wc[l];
  }
  const int xrow = (8 * wave + lr) * k32;
  // What stands behind the contraction's end (in its last unit, and in units past
  // it) becomes zeros on both sides: the next row's infinities and NaN stay out.
  auto copy_x = [&](uint8_t* to, int u) {
    const int q = (u0 + u) * kUnit;
#pragma unroll
    for (int l = 0; l < LX; ++l) {
      const int at = xc[l] < k32 - q ? xrow + xc[l] : kNowhere;
      copy_1k(xr, to + (group * BM / 8 + l * kWaves + wave) * 1024, at + (8 * l * kWaves * k32 + q));
    }
  };
  auto copy_w = [&](uint8_t* to, int u) {
    const int q = (u0 + u) * kUnit;
#pragma unroll
    for (int l = 0; l < LW; ++l) {
      // a gated weight's rows are whole units
      const bool in = kGated ? u0 + u < units : wc[l] < k32 - q;
      copy_1k(kGated && !kEven && (l & 1) ? ur : wr, to + (group * BN / 8 + l * kWaves + wave) * 1024,
              (in ? wo[l] : kNowhere) + (8 * (kGated ? l * kWaves >> 1 : l * kWaves) * k32 + q));
    }
  };
  // Fragments of a unit's first or second 64 codes. Token tile t reads rows
  // 16 t + i; channel tile t rows 64 (t / 4) + 16 (i / 4) + 4 (t % 4) + i % 4,
  // which leaves a lane with runs of 16 neighbouring channels. Both keys are
  // i / 2.
  const int xa = (group * BM + wm * TM * 16 + i) * kUnit;
  const int wa = (group * BN + wn * TN * 16 + 16 * (i >> 2) + (i & 3)) * kUnit;
  const int place[2] = {16 * (h ^ (i >> 1)), 16 * ((4 + h) ^ (i >> 1))};
  u32x4 fx[2][TM], fw[2][TN];
  auto read = [&](const uint8_t* x, const uint8_t* w, int half) {
#pragma unroll
    for (int t = 0; t < TN; ++t)
      fw[half][t] = ld16(w + wa + place[half] + (t >> 2) * (64 * kUnit) + (t & 3) * (4 * kUnit));
#pragma unroll
    for (int t = 0; t < TM; ++t) fx[half][t] = ld16(x + xa + place[half] + t * (16 * kUnit));
  };
  f32x4 acc[TM][TN];
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int half) {
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int b = 0; b < TN; ++b) acc[a][b] = mma16<kF16>(fw[half][b], fx[half][a], acc[a][b]);
  };
  // Unit u, whose first half's fragments are in registers: its second half is
  // read while the first is multiplied; then the next unit has to be whole,
  // its first half is read and this unit's parts filled again while the second
  // is multiplied. One barrier a unit.
  auto unit = [&](int u, uint8_t* x, uint8_t* w, const uint8_t* next_x, const uint8_t* next_w) {
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
      uint8_t* at = ring[1 + 2 * ((gr - 1) / (kFit > 0 ? kFit : 1))] + (gr - 1) % (kFit > 0 ? kFit : 1) * (BM * BN * 4);
      return reinterpret_cast<f32x4*>(at) + wave * (TM * TN * 64) + lane;
    };
#pragma unroll
    for (int gr = 1; gr < KS; ++gr) {
      if (group != gr) continue;
      f32x4* to = sums(gr);
#pragma unroll
      for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b) to[(a * TN + b) * 64] = acc[a][b];
    }
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int gr = 1; gr < KS; ++gr) {
      const f32x4* from = sums(gr);
#pragma unroll
      for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b) acc[a][b] += from[(a * TN + b) * 64];
    }
  }

  // The adapter's slots as more contraction, in terms that hold all bits of the float32
  // H or dH, operands straight from memory. Fragment rows as in the ring; tokens past the
  // last are not stored, channels past it are zeros.
  for (int ks = 0; ks < g.rpad / 32; ++ks) {
    // two terms in registers at a time, a part of one beside a widened fp16 B: more spill in the largest tiles
    constexpr int kFirst = kF16 && TM == 8 ? 4 : TM;
    u32x4 xa[TM], xc[TM];
    auto load = [&](u32x4(&to)[TM], int q, int first, int last) {
#pragma unroll
      for (int a = first; a < last; ++a) {
        const int64_t m = m0 + wm * TM * 16 + 16 * a + i;
        to[a] = ld16(g.ha + (m < g.m ? m : g.m - 1) * (3 * g.rpad) + q * g.rpad + 32 * ks + 8 * h);
      }
    };
    load(xa, 0, 0, TM);
    Wide<kF16> wb[TN];
#pragma unroll
    for (int b = 0; b < TN; ++b) {
      const int row = wn * TN * 16 + 64 * (b >> 2) + 16 * (i >> 2) + 4 * (b & 3) + (i & 3);
      const bool up = kGated && (row & 8) != 0;
      const int64_t n = n0 + (kGated ? 8 * (row >> 4) + (row & 7) : row);
      wb[b].t[0] = n < g.n ? ld8_bf16_window(g.hb + (n + (up ? g.up : 0)) * g.hb_ld, 32 * ks + 8 * h - (up ? g.shift : 0),
                                             g.hb_lim, (g.hb_ld % 8) == 0)
                           : u32x4{0, 0, 0, 0};
    }
    load(xc, 1, 0, kFirst);
#pragma unroll
    for (int b = 0; b < TN; ++b) wb[b] = widen<kF16>(wb[b].t[0]);
    auto multiply = [&](const u32x4(&x)[TM], int q) {
#pragma unroll
      for (int b = 0; b < TN; ++b)
#pragma unroll
        for (int a = 0; a < TM; ++a) acc[a][b] = mma_term<kF16>(wb[b], x[a], q, acc[a][b]);
    };
    multiply(xa, 0);
    __builtin_amdgcn_sched_barrier(0);
    load(xc, 1, kFirst, TM);
    load(xa, 2, 0, TM);
    multiply(xc, 1);
    multiply(xa, 2);
  }

  // Lane: tokens 16 a + i, channels 64 (b / 4) + 16 h + 4 (b % 4) + v: runs of 16
  // neighbouring channels (gated: of 8 outputs), 64 (32) the four lanes of a token.
  // n is a multiple of 16, so a run is whole or absent.
#pragma unroll
  for (int c = 0; c < TN / 4; ++c) {
    const int64_t nc = kGated ? n0 + wn * TN * 8 + 32 * c + 8 * h : n0 + wn * TN * 16 + 64 * c + 16 * h;
    if (nc >= g.n) continue;
#pragma unroll
    for (int a = 0; a < TM; ++a) {
      const int64_t m = m0 + wm * TM * 16 + 16 * a + i;
      if (m >= g.m) continue;
      const f32x4* s = acc[a] + 4 * c;
      u32x2 w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) w[b] = u32x2{cvt_16x2<kF16>(s[b][0], s[b][1]), cvt_16x2<kF16>(s[b][2], s[b][3])};
      if (!kGated || g.y != nullptr) {
        uint16_t* y = g.y + m * g.ldy + nc;
        st16(y, u32x4{w[0][0], w[0][1], w[1][0], w[1][1]});
        st16(kGated ? y + g.up : y + 8, u32x4{w[2][0], w[2][1], w[3][0], w[3][1]});
      }
      if (kGated) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int b = e >> 1, v = 2 * (e & 1);
          o[e] = cvt_16x2<kF16>(act_value<false>(s[b][v], g.act) * s[2 + b][v],
                                act_value<false>(s[b][v + 1], g.act) * s[2 + b][v + 1]);
        }
        st16(g.p + m * g.up + nc, u32x4{o[0], o[1], o[2], o[3]});
      }
    }
  }
}

template <int I, bool kGated>
hipError_t launch_tiles(const DenseArgs& g, bool f16, hipStream_t s) {
  constexpr Shape t = kShapes[I];
  constexpr int BM = t.bm, BN = t.bn, WM = t.wm, WN = t.wn, KS = t.groups, P = t.parts, BO = kGated ? BN / 2 : BN;
  const int tiles_m = static_cast<int>((g.m + BM - 1) / BM), tiles_n = static_cast<int>((g.n + BO - 1) / BO);
  auto kern = f16 ? dense_kernel<BM, BN, WM, WN, KS, P, true, kGated> : dense_kernel<BM, BN, WM, WN, KS, P, false, kGated>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tiles_m) * tiles_n), dim3(t.threads()), 0, s, g, tiles_m, tiles_n);
  return hipGetLastError();
}

template <bool kGated>
hipError_t launch_shape(int shape, const DenseArgs& g, bool f16, hipStream_t s) {
  switch (shape) {
    case 0:
      return launch_tiles<0, kGated>(g, f16, s);
    case 1:
      return launch_tiles<1, kGated>(g, f16, s);
    case 2:
      return launch_tiles<2, kGated>(g, f16, s);
    case 3:
      return launch_tiles<3, kGated>(g, f16, s);
    case 4:
      return launch_tiles<4, kGated>(g, f16, s);
    case 5:
      return launch_tiles<5, kGated>(g, f16, s);
    case 6:
      return launch_tiles<6, kGated>(g, f16, s);
  }
  return hipErrorInvalidValue;  // dense_fits refuses these sizes
}

// The rules count weight rows, two of a gated output, and bytes of contraction.
template <bool kGated>
hipError_t launch_product(DenseArgs g, bool f16, hipStream_t s) {
  constexpr int kOf = kGated ? 2 : 1;
  const Pick one = pick_shape(g.m, kOf * g.n, g.kb);
  const int64_t cols = full_rounds(g.m, kOf * g.n, g.kb, one) / kOf;
  if (cols > 0) {
    const int64_t n = g.n;
    g.n = cols;
    const hipError_t e = launch_shape<kGated>(0, g, f16, s);
    if (e != hipSuccess) return e;
    g.w += cols * g.kb;
    if (g.hb != nullptr) g.hb += cols * g.hb_ld;
    if (g.y != nullptr) g.y += cols;
    if (kGated) g.p += cols;
    g.n = n - cols;
    return launch_shape<kGated>(pick_shape(g.m, kOf * g.n, g.kb).shape, g, f16, s);
  }
  return launch_shape<kGated>(one.shape, g, f16, s);
}

// ---------------------------------------------------------------------------
// What a product over the restored weight needs beside its inputs, in one launch: the
// weight (or its transpose) in 16 bits, and the adapter's narrow product, H = X A^T or
// dH = s dY B, whose workgroups come first and end under the weight's memory traffic.
// In launches of their own H took 12 us of a 2048 x 22016 x 4096 call and 8 of 27 us of
// a 333 x 5120 x 1088 one.
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;    // with the transpose
constexpr int kRowThreads = 1024;  // of the weight as it is stored

// out32[i][j] = scale sum_q p[i][q] w(j, q), terms (m x 3 rpad) = scale2 out32 as terms
// with zeros behind the slots. w: slots x q, or (kCols) q x rpart, where slot j is column j mod
// rpart of part j / rpart's rows and zero in the others'.
struct Narrow {
  const uint16_t* p;
  int64_t m, q;
  const uint16_t* w;
  int slots, rpad;  // rpad: slots rounded up to 32; 0: none of this
  LoraParts parts;
  float scale, scale2;
  float* out32;
  uint16_t* terms;
};

// 16 tokens and 16 slots by a workgroup: its kW waves take units of 64 of the
// contraction (whole cache lines) in turn, operands straight from memory, and their sums
// meet in LDS in wave order. kCols: a lane's eight operands are strided, 2-byte loads.
// Bound by the lines that its loads touch, 16 for a kilobyte, at 16 bytes a cycle of its
// CU: 32 slots by a workgroup took 6.4 us for 1728 of contraction and 22 for 8128, and
// twice that for 64.
template <bool kF16, bool kCols, int kW>
__device__ __forceinline__ void narrow_tile(const Narrow& g, int64_t block, f32x4* red) {
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, h = lane >> 4, wave = tid >> 6;
  const int tiles = g.rpad / 16;
  const int64_t m0 = block / tiles * 16;
  const int slot = static_cast<int>(block % tiles) * 16 + i;
  if (slot - i >= g.slots) {  // zeros alone
    for (int o = wave; o < 4; o += kW)
      if (m0 + 4 * h + o < g.m) put_terms(g.terms + (m0 + 4 * h + o) * (3 * g.rpad), g.rpad, slot, 0.0f);
    return;
  }
  const uint16_t* prow = g.p + (m0 + i < g.m ? m0 + i : g.m - 1) * g.q;
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t u = wave; u < (g.q + 63) / 64; u += 2 * kW) {
    u32x4 pv[4], wv[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // halves of units u and u + kW
      const int64_t q = 64 * (u + kW * (c >> 1)) + 32 * (c & 1) + 8 * h;
      const bool in = q < g.q;  // q is a multiple of 16 long: a run of 8 is whole or absent
      const int64_t at = in ? q : 0;
      pv[c] = ld16(prow + at);
      if (!in) pv[c] = u32x4{0, 0, 0, 0};
      if constexpr (!kCols) {
        wv[c] = ld16(g.w + static_cast<int64_t>(slot < g.slots ? slot : 0) * g.q + at);
      } else {
        int part = 0;
#pragma unroll
        for (int l = 0; l < 3; ++l) part += (l + 1 < g.parts.g && at >= g.parts.end[l]) ? 1 : 0;
        const int col = slot - part * g.parts.rpart;
        const bool own = col >= 0 && col < g.parts.rpart;
        const uint16_t* w = g.w + at * g.parts.rpart + (own ? col : 0);
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = w[e * g.parts.rpart];
#pragma unroll
        for (int e = 0; e < 4; ++e) wv[c][e] = own ? v[2 * e] | v[2 * e + 1] << 16 : 0u;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) acc = mma16<kF16>(pv[c], wv[c], acc);
  }
  red[wave * 64 + lane] = acc;
  __syncthreads();
  // acc[v]: token 4 h + v, slot
  const float* rf = reinterpret_cast<const float*>(red);
  for (int v = wave; v < 4; v += kW) {
    const int64_t m = m0 + 4 * h + v;
    if (m >= g.m) continue;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kW; ++w) sum += rf[(w * 64 + lane) * 4 + v];
    sum = slot < g.slots ? g.scale * sum : 0.0f;
    if (g.out32 != nullptr && slot < g.slots) g.out32[m * g.slots + slot] = sum;
    put_terms(g.terms + m * (3 * g.rpad), g.rpad, slot, g.scale2 * sum);
  }
}

// The weight as it is stored, n x k: a thread takes words of eight codes, so that the
// lanes of a store write neighbouring 16 bytes.
constexpr int kWords = 4;

template <bool kDQ, bool kF16>
__global__ __launch_bounds__(kRowThreads) void restore_kernel(PackedW w, uint16_t* out, Levels L, int narrow_blocks,
                                                              Narrow g) {
  constexpr int kThreads = kRowThreads;
  __shared__ f32x4 red[kThreads];
  if (static_cast<int>(blockIdx.x) < narrow_blocks) {
    narrow_tile<kF16, false, kThreads / 64>(g, blockIdx.x, red);
    return;
  }
  const int64_t words = w.n * w.k / 8;  // a multiple of 128
  const int64_t first = static_cast<int64_t>(blockIdx.x - narrow_blocks) * (kWords * kThreads) + threadIdx.x;
  uint32_t c[kWords], code[kWords];
  float value[kWords];
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const int64_t at = first + j * kThreads < words ? first + j * kThreads : words - 1;
    c[j] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(w.codes) + at);
    const int64_t block = at / 8;
    code[j] = kDQ ? w.scale_codes[block] : 0;
    value[j] = kDQ ? w.group_scale[block / 256] : w.absmax[block];
  }
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const BlockLut lut = make_block_lut<kF16>(L.v, kDQ ? dq_unit(code[j], w.dq) * value[j] : value[j]);
    uint32_t v[4];
    lut8_natural_order(lut, c[j], v);
    const int64_t at = first + j * kThreads;
    if (at < words) st16(out + at * 8, u32x4{v[0], v[1], v[2], v[3]});
  }
}

// The weight's transpose, k x n. A workgroup takes 64 weight rows and 4 of their
// 64-weight blocks: a lane restores one block of one row and writes it down LDS
// columns, which leave as whole 128-byte runs. A^T for the product's adapter slots is
// made here too, and where dH is not, B^T.
constexpr int kTrRows = 64, kTrBlocks = 4;
constexpr int kTrLd = kTrRows + 8;  // elements of an LDS row: 16-byte reads stay aligned, rows shift by 4 banks

template <bool kDQ, bool kF16>
__global__ __launch_bounds__(kThreads) void restore_t_kernel(PackedW w, uint16_t* out, Levels L, int narrow_blocks,
                                                             Narrow g, const uint16_t* a, uint16_t* at, uint16_t* bt,
                                                             int tr_blocks) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[kTrBlocks * 64 * kTrLd];
  static_assert(kTrTile <= kTrBlocks * 64 * kTrLd && 4 * 64 * 16 <= sizeof(tile), "all use the tile");
  if (static_cast<int>(blockIdx.x) < narrow_blocks) {
    narrow_tile<kF16, true, 4>(g, blockIdx.x, reinterpret_cast<f32x4*>(tile));
    return;
  }
  const int64_t id = blockIdx.x - narrow_blocks;
  if (id < tr_blocks) {  // the first k / 64 of its tiles are A's
    lora_transpose_tile(tile, id, a, g.w, w.n, w.k, g.slots, g.rpad, g.parts, at, bt);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t nbk = w.k / 64, tiles_k = (nbk + kTrBlocks - 1) / kTrBlocks;
  const int64_t n0 = (id - tr_blocks) / tiles_k * kTrRows, b0 = (id - tr_blocks) % tiles_k * kTrBlocks;
  const int64_t n = n0 + lane < w.n ? n0 + lane : w.n - 1, kb = b0 + wave < nbk ? b0 + wave : nbk - 1;
  const int64_t block = n * nbk + kb;
  const u32x4 c0 = ld16(w.codes + block * 32), c1 = ld16(w.codes + block * 32 + 16);
  const float s = kDQ ? dq_unit(w.scale_codes[block], w.dq) * w.group_scale[block / 256] : w.absmax[block];
  const BlockLut lut = make_block_lut<kF16>(L.v, s);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t v[4];
    lut8_natural_order(lut, j < 4 ? c0[j] : c1[j - 4], v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      tile[(wave * 64 + 8 * j + e) * kTrLd + lane] = static_cast<uint16_t>(e & 1 ? v[e >> 1] >> 16 : v[e >> 1]);
  }
  __syncthreads();
  // 8 lanes a row of 64
#pragma unroll
  for (int it = 0; it < kTrBlocks * 64 / 32; ++it) {
    const int row = 32 * it + (threadIdx.x >> 3), c = 8 * (threadIdx.x & 7);
    const int64_t k = b0 * 64 + row;
    if (k < w.k && n0 + c < w.n) st16(out + k * w.n + n0 + c, ld16(tile + row * kTrLd + c));  // n % 16 == 0: runs are whole
  }
}

int narrow_blocks(const Narrow& g) { return static_cast<int>((g.m + 15) / 16) * (g.rpad / 16); }

}  // namespace

hipError_t launch_dense_gated(const uint16_t* w16, int64_t n2, int64_t k, const uint16_t* x, int64_t m,
                              const uint16_t* hs, const uint16_t* b, int rpart, int rpad, int act, uint16_t* y,
                              uint16_t* p, hipStream_t st, bool f16) {
  const DenseArgs g{reinterpret_cast<const uint8_t*>(w16), reinterpret_cast<const uint8_t*>(x), m, n2 / 2, 2 * k, n2 / 2,
                    hs, b, rpart, rpart, rpad, rpart, y, n2, p, act};
  return launch_product<true>(g, f16, st);
}

hipError_t launch_restore(const PackedW& w, uint16_t* w16, const uint16_t* x, int64_t m, const uint16_t* a, int slots,
                          int rpad, float s, float* h32, uint16_t* hs, hipStream_t st, bool f16) {
  const Narrow g{x, m, w.k, a, slots, rpad, LoraParts{}, 1.0f, s, h32, hs};
  const int first = narrow_blocks(g);
  const int64_t grid = first + (w.n * w.k / 8 + kWords * kRowThreads - 1) / (kWords * kRowThreads);
  auto kern = f16 ? (w.dq ? restore_kernel<true, true> : restore_kernel<false, true>)
                  : (w.dq ? restore_kernel<true, false> : restore_kernel<false, false>);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(kRowThreads), 0, st, w, w16,
                     codebook_table(w.codebook), first, g);
  return hipGetLastError();
}

hipError_t launch_restore_t(const PackedW& w, uint16_t* wt16, const uint16_t* dy, int64_t m, const uint16_t* a,
                            const uint16_t* b, int slots, int rpad, const LoraParts* parts, float s, float* dh32,
                            uint16_t* dhs, uint16_t* at, uint16_t* bt, hipStream_t st, bool f16) {
  LoraParts one;
  one.rpart = slots;
  one.end[0] = static_cast<int>(w.n);
  const Narrow g{dy, m, w.n, b, slots, rpad, parts != nullptr ? *parts : one, s, 1.0f, dh32, dhs};
  const bool narrow = dense_narrow(w.n);
  const int first = narrow ? narrow_blocks(g) : 0;
  const int tr_blocks = rpad == 0                     ? 0
                        : !narrow                     ? static_cast<int>(lora_transpose_tiles(w.n, w.k))
                        : wt16 != nullptr             ? static_cast<int>(w.k / kTrCols)
                                                      : 0;
  const int64_t weight = (w.n + kTrRows - 1) / kTrRows * ((w.k / 64 + kTrBlocks - 1) / kTrBlocks);
  const int64_t grid = first + tr_blocks + (wt16 != nullptr ? weight : 0);
  auto kern = f16 ? (w.dq ? restore_t_kernel<true, true> : restore_t_kernel<false, true>)
                  : (w.dq ? restore_t_kernel<true, false> : restore_t_kernel<false, false>);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, st, w, wt16,
                     codebook_table(w.codebook), first, g, a, at, bt, tr_blocks);
  return hipGetLastError();
}

hipError_t launch_dense_dx(const uint16_t* wt16, int64_t n, int64_t k, const uint16_t* dy, int64_t m,
                           const uint16_t* dhs, const uint16_t* at, int rpad, uint16_t* dx, hipStream_t st, bool f16) {
  const DenseArgs g{reinterpret_cast<const uint8_t*>(wt16), reinterpret_cast<const uint8_t*>(dy), m, k, 2 * n, 0,
                    dhs, at, rpad, rpad, rpad, 0, dx, k, nullptr, 0};
  return launch_product<false>(g, f16, st);
}

}  // namespace qlora
