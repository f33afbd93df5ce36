// Both adapter gradients of a linear whose input was kept as 8-bit rows:
//   dA = dH^T X, X[m][c] = code[m][c] scale[m]  (slots x k)
//   dB = s dY^T H                               (n x r)
// as one launch over two problems out[j][c] = sum_m U[m][j] V[m][c], U float32
// (dH times the row's scale; H) and V the codes (exact in bf16) or dY.
//
// Bound by reading V once: k + 2 n bytes a token. 2048 tokens, rank 16: k = 11008, n =
// 4096 holds 39 MB and takes 13.7 us (2.9 TB/s), and 5 for the sums of two splits; k =
// 4096, n = 22016 in two parts 99 MB in 25 us (4.0 TB/s). With what a step computes from
// its loads in front of the step before it, whose loads then wait for it, 25 us for 14.
// Above rank 16 V is read once for every 32 slots of a part (codes for every 32 of all):
// the first size takes 19 us at rank 32, 30 at 64 and 56 at 128, the second 31 and 54 at
// 32 and 64; with both steps' U in registers, which spills, 27, 45, 86, 48 and 66, and 16
// slots at a time 21, 39, 75, 42 and 86.
//
// Matrix cores in bf16 with float32 sums (v_mfma_f32_16x16x32_bf16), every
// float32 U split into three bf16 terms that hold all of its 24 bits (the low 16
// bits cut off twice, the rest rounded); an fp16 dY is split into two, its upper
// eight bits and the other three, both exact. So no product is rounded, and the
// gradients are float32 sums. The extra products are free next to the memory.
//
// No LDS on the way in: a contraction step is 32 rows; lane (i, g) loads 8 columns
// of rows 8 g .. 8 g + 7 (whole 128- or 256-byte runs of a row for its 16 lanes)
// and element t of the 8 rows is its operand for the tile of columns 8 i + t.
// A workgroup takes 128 columns and 16 or 32 slots; its eight waves take the
// steps of its rows in turn, and their sums meet in LDS in wave order. Few columns
// are split over the rows as well, into partial sums that are added in order by a
// second launch; results repeat bit for bit.
#include <type_traits>

#include "internal.h"
#include "mfma.h"

namespace qlora {
namespace {

constexpr int kCols = 128, kRows = 32, kWaves = 8, kThreads = 64 * kWaves;

enum VKind { kCodes, kBf16, kHalf };

struct Problem {
  const float* u;       // m x ldu
  const float* uscale;  // m, or null
  const void* v;        // m x ldv
  float* out;           // splits x slots x cn partial sums (one split: dA itself)
  float* db;            // one split: cn x slots, times scale
  float scale;
  int64_t cn, ldv;
  int ldu;
  int slots;  // of a column
  int strips, tiles;  // workgroups along the columns and the slots
  LoraParts lp;       // dB of grouped weights: a column's part owns slots from part rpart on
};

// Eight rows' 8 columns as loaded.
template <int kKind>
struct Block {
  typedef typename std::conditional<kKind == kCodes, u32x2, u32x4>::type Word;
  Word w[8];
};

// Element t of the eight rows as bf16 pairs; kHalf: its upper bits, and in `low`
// the rest.
template <int kKind>
__device__ __forceinline__ u32x4 operand(const Block<kKind>& b, int t, u32x4* low) {
  uint32_t hi[4], lo[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (kKind == kCodes) {
      const float f0 = static_cast<float>(static_cast<int8_t>(b.w[2 * e][t >> 2] >> (8 * (t & 3))));
      const float f1 = static_cast<float>(static_cast<int8_t>(b.w[2 * e + 1][t >> 2] >> (8 * (t & 3))));
      hi[e] = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);  // exact: 8 bits
    } else if constexpr (kKind == kBf16) {
      hi[e] = __builtin_amdgcn_perm(b.w[2 * e + 1][t >> 1], b.w[2 * e][t >> 1], (t & 1) ? 0x07060302u : 0x05040100u);
    } else {
      const uint32_t w0 = b.w[2 * e][t >> 1], w1 = b.w[2 * e + 1][t >> 1];
      const float f0 = (t & 1) ? hi16<true>(w0) : lo16<true>(w0), f1 = (t & 1) ? hi16<true>(w1) : lo16<true>(w1);
      hi[e] = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x07060302u);
      const float l0 = f0 - __uint_as_float(__float_as_uint(f0) & 0xFFFF0000u);
      const float l1 = f1 - __uint_as_float(__float_as_uint(f1) & 0xFFFF0000u);
      lo[e] = __builtin_amdgcn_perm(__float_as_uint(l1), __float_as_uint(l0), 0x07060302u);
    }
  }
  if (kKind == kHalf) *low = u32x4{lo[0], lo[1], lo[2], lo[3]};
  return u32x4{hi[0], hi[1], hi[2], hi[3]};
}

// The three bf16 terms of eight float32.
struct Terms {
  u32x4 t[3];
};
__device__ __forceinline__ Terms split3(const float* u) {
  Terms r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t h[2], m[2], l[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float f = u[2 * e + q];
      h[q] = __float_as_uint(f);
      const float f1 = f - __uint_as_float(h[q] & 0xFFFF0000u);
      m[q] = __float_as_uint(f1);
      l[q] = f32_to_bf16_rne(f1 - __uint_as_float(m[q] & 0xFFFF0000u));
    }
    r.t[0][e] = __builtin_amdgcn_perm(h[1], h[0], 0x07060302u);
    r.t[1][e] = __builtin_amdgcn_perm(m[1], m[0], 0x07060302u);
    r.t[2][e] = l[0] | l[1] << 16;
  }
  return r;
}

template <int kKind, int RT>
__device__ __forceinline__ void solve(const Problem& p, int64_t M, int id, int splits, int64_t per, f32x4* red) {
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = id % splits, tile = id / splits % p.tiles, strip = id / splits / p.tiles;
  const int64_t c0 = static_cast<int64_t>(strip) * kCols;
  const int j0 = tile * 16 * RT;
  int part = 0;
#pragma unroll
  for (int l = 0; l < 3; ++l) part += (l + 1 < p.lp.g && c0 >= p.lp.end[l]) ? 1 : 0;
  const float* u = p.u + part * p.lp.rpart;
  const int64_t mb = split * per, me = mb + per < M ? mb + per : M;

  const int64_t col = c0 + 8 * i < p.cn ? c0 + 8 * i : 0;  // cn % 16 == 0; columns past it are not stored
  f32x4 acc[RT][8];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[a][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // A step's operands as loaded; nothing is computed from them before the step, so
  // that the next one's loads are in flight under it. Rows past the last are read
  // from it and multiplied by zeros. With 32 slots U, which stays in L2, is loaded at the
  // step itself: two steps of it leave no registers, and a spilled load has to arrive
  // before it can be stored, in front of the step that it should be in flight under.
  typedef typename Block<kKind>::Word Word;
  struct Slots {
    float u[RT][8], scale[kKind == kCodes ? 8 : 1];
  };
  struct Step {
    Block<kKind> b;
    Slots s;
  };
  constexpr bool kAhead = RT == 1;
  auto row_of = [&](int64_t m0, int e) {
    const int64_t m = m0 + 8 * g + e;
    return m < M ? m : M - 1;
  };
  auto load_slots = [&](int64_t m0, Slots& s) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t mr = row_of(m0, e);
      if (kKind == kCodes) s.scale[e] = p.uscale[mr];
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        const int j = j0 + 16 * a + i;
        s.u[a][e] = u[mr * p.ldu + (j < p.slots ? j : 0)];
      }
    }
  };
  auto load = [&](int64_t m0, Step& s) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const char* row = static_cast<const char*>(p.v) + (row_of(m0, e) * p.ldv + col) * (kKind == kCodes ? 1 : 2);
      s.b.w[e] = *reinterpret_cast<const Word*>(row);
    }
    if (kAhead) load_slots(m0, s.s);
  };
  auto multiply = [&](int64_t m0, Step& s) {
    if (!kAhead) load_slots(m0, s.s);
    Terms terms[RT];
#pragma unroll
    for (int a = 0; a < RT; ++a) {
      float uv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        uv[e] = m0 + 8 * g + e < me && j0 + 16 * a + i < p.slots
                    ? (kKind == kCodes ? s.s.u[a][e] * s.s.scale[e] : s.s.u[a][e])
                    : 0.0f;
      terms[a] = split3(uv);
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      u32x4 low;
      const u32x4 v = operand<kKind>(s.b, t, &low);
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          acc[a][t] = mma16<false>(terms[a].t[q], v, acc[a][t]);
          if (kKind == kHalf) acc[a][t] = mma16<false>(terms[a].t[q], low, acc[a][t]);
        }
      if (t % 2 == 1) __builtin_amdgcn_sched_barrier(0);  // two operands in registers at a time, not all eight
    }
  };
  constexpr int kStride = kWaves * kRows;
  Step s0, s1;
  int64_t m0 = mb + wave * kRows;
  if (m0 < me) load(m0, s0);
  for (; m0 < me; m0 += 2 * kStride) {
    if (m0 + kStride < me) load(m0 + kStride, s1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(m0, s0);
    __builtin_amdgcn_sched_barrier(0);
    if (m0 + kStride >= me) break;
    if (m0 + 2 * kStride < me) load(m0 + 2 * kStride, s0);
    __builtin_amdgcn_sched_barrier(0);
    multiply(m0 + kStride, s1);
    __builtin_amdgcn_sched_barrier(0);
  }

  // acc[a][t][v]: slot j0 + 16 a + 4 g + v, column c0 + 8 i + t. Thread q sums
  // slot q / 32, columns 4 (q % 32) .. + 3 of each 16 slots over the waves.
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int t = 0; t < 8; ++t) red[((wave * RT + a) * 8 + t) * 64 + lane] = acc[a][t];
  __syncthreads();
  const float* rf = reinterpret_cast<const float*>(red);
  const int slot = tid >> 5, c4 = 4 * (tid & 31);
  const int64_t c = c0 + c4;
  if (c >= p.cn) return;
#pragma unroll
  for (int a = 0; a < RT; ++a) {
    const int j = j0 + 16 * a + slot;
    if (j >= p.slots) continue;
    f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sum[e] += rf[(((w * RT + a) * 8 + ((c4 + e) & 7)) * 64 + 16 * (slot >> 2) + (c4 >> 3)) * 4 + (slot & 3)];
    if (p.db != nullptr) {
#pragma unroll
      for (int e = 0; e < 4; ++e) p.db[(c + e) * p.slots + j] = p.scale * sum[e];
    } else {
      *reinterpret_cast<f32x4*>(p.out + (static_cast<int64_t>(split) * p.slots + j) * p.cn + c) = sum;
    }
  }
}

template <bool kF16, int RT>
__global__ __launch_bounds__(kThreads) void rank_grad8_kernel(Problem pa, Problem pb, int64_t M, int splits, int64_t per) {
  __shared__ f32x4 red[kWaves * RT * 8 * 64];
  const int id = blockIdx.x, first = pa.strips * pa.tiles * splits;
  if (id < first) solve<kCodes, RT>(pa, M, id, splits, per, red);
  else solve<kF16 ? kHalf : kBf16, RT>(pb, M, id - first, splits, per, red);
}

// da[j][c] = sum over splits of part0[s][j][c]; db[c][j] = scale times that of
// part1, both in split order.
__global__ __launch_bounds__(256) void rank_grad8_final_kernel(const float* part0, const float* part1, int64_t na,
                                                               int64_t n, int r, int splits, float scale, float* da,
                                                               float* db) {
  const int64_t nb = n * r;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= na + nb) return;
  const bool second = idx >= na;
  const float* part = second ? part1 + (idx - na) : part0 + idx;
  const int64_t step = second ? nb : na;
  float sum = 0.0f;
  for (int s = 0; s < splits; ++s) sum += part[s * step];
  if (!second) {
    da[idx] = sum;
    return;
  }
  const int64_t j = (idx - na) / n, c = (idx - na) % n;
  db[c * r + j] = scale * sum;
}

// 16-slot tiles of a workgroup, by the rank of a part: grouped calls read the codes
// once for every 16 of their slots, which are few next to dY.
int slot_tiles(int r) { return r > 16 ? 2 : 1; }

int tiles_of(int slots, int rt) { return (slots + 16 * rt - 1) / (16 * rt); }
int64_t workgroups(int64_t n, int64_t k, int slots, int r) {
  return (k + kCols - 1) / kCols * tiles_of(slots, slot_tiles(r)) + (n + kCols - 1) / kCols * tiles_of(r, slot_tiles(r));
}

}  // namespace

int rank_grad8_splits(int64_t m, int64_t n, int64_t k, int slots, int r) {
  // About a workgroup a CU, a step at least for each of its waves. 2048 tokens, n = 4096,
  // k = 11008: 13.7 us with two splits, 16.1 with four; k = 4096, n = 22016 in two parts:
  // 25 us and no second launch with one, 26 and 6 with two.
  int64_t s = 256 / workgroups(n, k, slots, r);
  const int64_t by_rows = m / (kWaves * kRows);
  if (s > by_rows) s = by_rows;
  if (s > 16) s = 16;
  return static_cast<int>(s < 1 ? 1 : s);
}

hipError_t launch_rank_grads8(const float* dh, const int8_t* x, int64_t ldx, const float* xscale, int64_t k,
                              const float* h, const uint16_t* dy, int64_t n, int64_t m, int slots,
                              const LoraParts* parts, float scale, float* part, float* da, float* db, hipStream_t st,
                              bool f16) {
  const int r = parts != nullptr ? parts->rpart : slots;
  const int splits = rank_grad8_splits(m, n, k, slots, r);
  const int64_t per = ((m + splits - 1) / splits + kRows - 1) / kRows * kRows;
  float* part1 = part + static_cast<int64_t>(splits) * slots * k;
  auto strips = [](int64_t c) { return static_cast<int>((c + kCols - 1) / kCols); };
  const Problem pa{dh, xscale, x, splits == 1 ? da : part, nullptr, 1.0f, k, ldx, slots, slots, strips(k),
                   tiles_of(slots, slot_tiles(r)), LoraParts{}};
  const Problem pb{h, nullptr, dy, part1, splits == 1 ? db : nullptr, scale, n, n, slots, r, strips(n),
                   tiles_of(r, slot_tiles(r)), parts != nullptr ? *parts : LoraParts{}};
  const unsigned grid = static_cast<unsigned>(workgroups(n, k, slots, r) * splits);
  auto kern = slot_tiles(r) == 1 ? (f16 ? rank_grad8_kernel<true, 1> : rank_grad8_kernel<false, 1>)
                                 : (f16 ? rank_grad8_kernel<true, 2> : rank_grad8_kernel<false, 2>);
  hipLaunchKernelGGL(kern, dim3(grid), dim3(kThreads), 0, st, pa, pb, m, splits, per);
  if (splits > 1) {
    const int64_t na = static_cast<int64_t>(slots) * k, total = na + n * r;
    hipLaunchKernelGGL(rank_grad8_final_kernel, dim3(static_cast<unsigned>((total + 255) / 256)), dim3(256), 0, st,
                       part, part1, na, n, r, splits, scale, da, db);
  }
  return hipGetLastError();
}

}  // namespace qlora
