// Decode path of the gated feed-forward block, 1 to 16 tokens a launch: P = act(G) U with
// [G | U] = X W16^T + s [H_1 B_1^T | H_2 B_2^T], W read straight from its packed
// NF4 form in one pass.
//
// Bound by the vector instructions that restore the packed weight (0.516 bytes a weight):
// over a 44032 x 8192 weight they take 59% of the SIMDs' cycles (3.0 a weight, addresses
// included), the matrix cores 10%, LDS is active for 29%, and a wave waits for 46% of its
// own, so the stream stands at 3.1 TB/s however long it is:
//   * the 16 levels are expanded into an LDS table over a code byte, entry e the
//     float32 levels of its two nibbles, stored 32 times so that the lanes of a read
//     hit different banks. A byte permute, one 8-byte read, two products with the
//     block's scale and one conversion restore two weights exactly as
//     bf16(fl32(L s)): 2 vector instructions a weight, where a table of the block's
//     own 16 values in registers takes 3.4;
//   * the products run on the matrix cores, tokens padded to 16. A workgroup takes
//     groups of 16 weight rows, 8 of gate and the 8 of up of the same outputs; its
//     16 waves hold a slice of 256 k of X in registers for all of them, lane (i, g)
//     restoring block g of the slice of row i;
//   * codes come through LDS, three groups ahead, in copies of whole 128-byte runs:
//     loaded straight into the lanes that restore them each load touches 16 lines
//     for a kilobyte, and the loads' addresses bound the kernel (21.5 us);
//   * the sums of six groups meet in LDS at once, in wave order: results do not
//     depend on scheduling.
// H comes from a kernel of its own: formed in every workgroup it would read all of
// A 256 times.
// One token, 22016 x 4096 (46.5 MB): 16.0 us alone (2.9 TB/s; 10 at a copy's rate), 18.4
// with H, 16 tokens 17.8 and 21.9; 1024 x 1024 without an adapter 5.9, of which the
// start, the table and the end are most. 44032 x 8192 (186 MB) in two passes and two
// batches: 59.5. The row kernels of one or two tokens (gemv_kernels.hip), which multiply
// by a 16-bit level and scale afterwards, take 11.5 and 45.8 for these weights.
#include <type_traits>

#include "bufmem.h"
#include "gate.h"
#include "internal.h"
#include "mfma.h"
#include "nf4_lut.h"

namespace qlora {
namespace {

constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int kGroups = 6;                        // row groups of a batch, whose sums meet at once
constexpr int kAhead = 3;                         // of them, copies in flight
constexpr int kTable = 256 * 32 * 8;              // bytes: code bytes x copies x two levels
constexpr int kPart = 16 * 128;                   // a wave's 256 k of a group's codes
constexpr int kSlot = kWaves * kPart;             // a slot of the ring
constexpr int kRegion = 8 * 512;                  // a wave's 256 k of 8 tokens
constexpr int kStage = kWaves * kRegion;          // of the workgroup
static_assert(kSlot == 2 * kWaves * 1024 && kGroups == 2 * kAhead, "two groups' sums go where a slot's codes were");
static_assert(kStage == kTable && kStage == 2 * kSlot && kAhead == 3, "X stands where the table, and codes, follow");
static_assert(kGroups <= kWaves && kTable + kAhead * kSlot <= 160 * 1024, "one wave sums a group");

struct Args {
  PackedW w;
  const uint16_t* x;
  int M;
  const float* h;     // M x 2 rb, or null
  const uint16_t* b;  // n x rb
  int rb;
  float s;
  uint16_t* y;        // M x n, or null
  uint16_t* p;        // M x n / 2
  int act;
  Levels L;
};

__device__ __forceinline__ float level(const Levels& L, int c) {
  float v = L.v[0];
#pragma unroll
  for (int q = 1; q < 16; ++q) v = c == q ? L.v[q] : v;
  return v;
}

// A contraction step of H B^T, 32 slots: lane (i, g) holds eight of token i of H and
// of weight row i of B (0 where the row's part does not own the slot).
struct Slots {
  f32x4 h[2];
  u32x4 b;
};

// H's float32 in three bf16 terms, which hold all 24 bits, an fp16 B in two, which
// hold all 11, so no product is rounded.
template <bool kF16>
__device__ __forceinline__ f32x4 slot_products(const Slots& v, f32x4 acc) {
  u32x4 ht[3], bt[2];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t h[3][2], b[2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float f = v.h[e >> 1][2 * (e & 1) + q];
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        h[c][q] = __float_as_uint(f) >> 16;
        f -= __uint_as_float(h[c][q] << 16);
      }
      b[0][q] = q == 0 ? v.b[e] & 0xFFFFu : v.b[e] >> 16;
      b[1][q] = 0;
      if (kF16) {
        const float w = lo16<true>(b[0][q]);
        b[0][q] = __float_as_uint(w) >> 16;
        b[1][q] = __float_as_uint(w - __uint_as_float(b[0][q] << 16)) >> 16;
      }
    }
#pragma unroll
    for (int c = 0; c < 3; ++c) ht[c][e] = h[c][0] | h[c][1] << 16;
#pragma unroll
    for (int c = 0; c < 2; ++c) bt[c][e] = b[c][0] | b[c][1] << 16;
  }
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    acc = mma16<false>(ht[c], bt[0], acc);
    if (kF16) acc = mma16<false>(ht[c], bt[1], acc);
  }
  return acc;
}

// kLong: k > 4096, in passes of 4096 with a slice of X for each.
// kMany: over 8 tokens.
template <bool kDQ, bool kF16, bool kLong, bool kMany>
__global__ __launch_bounds__(kThreads) void gated_gemv_kernel(Args a) {
  __shared__ __attribute__((aligned(16))) unsigned char table[kTable];
  // one array a slot: the compiler can then tell a copy into one from what is read
  // out of another, and waits for none of them by itself
  __shared__ __attribute__((aligned(16))) unsigned char slot0[kSlot];
  __shared__ __attribute__((aligned(16))) unsigned char slot1[kSlot];
  __shared__ __attribute__((aligned(16))) unsigned char slot2[kSlot];
  unsigned char* const ring[kAhead] = {slot0, slot1, slot2};
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // 32-bit offsets: n k <= 2^31
  const int K = static_cast<int>(a.w.k), N = static_cast<int>(a.w.n), half = N / 2;
  const int nbk = K / 64, passes = kLong ? (nbk + 63) / 64 : 1;
  const int nrg = N / 16, grid = static_cast<int>(gridDim.x);
  const int mine = (nrg - static_cast<int>(blockIdx.x) + grid - 1) / grid;  // groups of this workgroup
  const int slots = 2 * a.rb;

  // group q of the workgroup: outputs 8 rg .. 8 rg + 7 (past its last: read, not used)
  auto group_of = [&](int q) {
    const int rg = static_cast<int>(blockIdx.x) + q * grid;
    return rg < nrg ? rg : nrg - 1;
  };
  // weight row i of a group: gate's for lanes 0 .. 7, up's of the same outputs for 8 .. 15
  const int lane_row = (i & 7) + (i >> 3) * half;

  // A group's codes of the wave's slice, 16 rows of 128 bytes, into a slot of the
  // ring: two copies of 8 rows (gate's, up's), lane l the 16 bytes at row l / 8 and
  // place l % 8; piece c of row r stands at place c ^ (r / 2 % 8). The scales follow
  // the copies, so what waits for them has the codes as well. All places are in the
  // weight or, behind its last row, read as zeros; blocks past the row's end meet
  // zeros of X.
  const __amdgpu_buffer_rsrc_t cr = make_rsrc(a.w.codes, static_cast<int64_t>(N) * (K / 2));
  const __amdgpu_buffer_rsrc_t sr = kDQ ? make_rsrc(a.w.scale_codes, static_cast<int64_t>(N) * nbk)
                                        : make_rsrc(a.w.absmax, static_cast<int64_t>(N) * nbk * 4);
  const __amdgpu_buffer_rsrc_t gr = make_rsrc(a.w.group_scale, kDQ ? (static_cast<int64_t>(N) * nbk + 255) / 256 * 4 : 0);
  int copy_at[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
    copy_at[t] = ((lane >> 3) + t * half) * (K / 2) + wave * 128 + 16 * ((lane & 7) ^ ((lane >> 4) + 4 * t));
  constexpr int kOps = kDQ ? 4 : 3;
  struct Scale {
    uint32_t code;
    float value;
  } sc[kAhead];
  // A wave whose slice lies behind the row's end has nothing to copy or multiply.
  auto live = [&](int pass) { return pass * 64 + 4 * wave < nbk; };
  auto stage = [&](int q, int pass, int slot) {
    if (!live(pass)) return;
    const int first = group_of(q) * 8;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(cr, (lds_void*)(ring[slot] + wave * kPart + t * 1024), 16,
                                               copy_at[t] + first * (K / 2) + pass * 2048, 0, 0, 0);
    }
    const int kb = pass * 64 + 4 * wave + g;
    const int block = (first + lane_row) * nbk + (kb < nbk ? kb : nbk - 1);
    if (kDQ) {
      sc[slot].code = __builtin_amdgcn_raw_buffer_load_b8(sr, block, 0, 0);
      sc[slot].value = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(gr, block / 256 * 4, 0, 0));
    } else {
      sc[slot].code = 0;
      sc[slot].value = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(sr, block * 4, 0, 0));
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // The lane, opaque to the compiler: addresses formed from it are formed anew in
  // every batch. Formed in front of the loop they are spilled, 50 MB of stores (6 us).
  auto fresh_lane = [&]() {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };

  // X: the wave's 256 k of 8 tokens, two tokens a copy; lane l moves the piece (16
  // bytes) that belongs at its place: piece p of row r stands at p ^ r. Tokens past
  // the last read zeros.
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, static_cast<int64_t>(a.M) * K * 2);
  auto copy_x = [&](unsigned char* to, int r0, int pass) {
    if (!live(pass)) return;
    const int lane = fresh_lane();
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int row = 2 * t + (lane >> 5);
      const int off = (r0 + row) * K * 2 + (pass * 64 + 4 * wave) * 128 + 16 * ((lane & 31) ^ row);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_void*)(to + t * 1024), 16, off, 0, 0, 0);
    }
  };
  u32x4 xa[8];
  auto read_x = [&](const unsigned char* from, int r0, int pass) {
    const int l = fresh_lane(), i = l & 15, g = l >> 4;
    if ((i & 8) != r0) return;
    const bool has = r0 + (i & 7) < a.M && pass * 64 + 4 * wave + g < nbk;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xa[j] = *reinterpret_cast<const u32x4*>(from + (i & 7) * 512 + 16 * ((8 * g + j) ^ (i & 7)));
      if (!has) xa[j] = u32x4{0, 0, 0, 0};
    }
  };

  // Slots j0 .. j0 + 31 of H and of B's rows of group q. Ranks that are multiples of
  // eight have a lane's slots in one part, and 16-byte loads.
  const bool wide = a.rb % 8 == 0;
  auto load_slots = [&](int q, int j0) {
    const int l = fresh_lane(), i = l & 15, g = l >> 4, lane_row = (i & 7) + (i >> 3) * half;
    Slots v;
    const int j = j0 + 8 * g, jb = j - (i >> 3) * a.rb;
    const float* hr = a.h + (i < a.M ? i : a.M - 1) * slots;
    const uint16_t* br = a.b + (group_of(q) * 8 + lane_row) * a.rb;
    if (wide) {
      v.h[0] = *reinterpret_cast<const f32x4*>(hr + (j < slots ? j : 0));
      v.h[1] = *reinterpret_cast<const f32x4*>(hr + (j < slots ? j : 0) + 4);
      v.b = ld16(br + (jb >= 0 && jb < a.rb ? jb : 0));
    } else {
      v.b = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v.h[e >> 2][e & 3] = hr[j + e < slots ? j + e : 0];
        const uint32_t w = br[jb + e >= 0 && jb + e < a.rb ? jb + e : 0];
        v.b[e >> 1] |= jb + e >= 0 && jb + e < a.rb ? w << (16 * (e & 1)) : 0u;
      }
    }
    return v;
  };
  // s H B^T of the group that this wave sums
  const int own = wave < kGroups ? wave : 0;
  auto adapter = [&](Slots v, int q) {
    const int l = fresh_lane(), i = l & 15, g = l >> 4;
    f32x4 lo = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < slots; j0 += 32) {
      if (j0 > 0) v = load_slots(q, j0);
      const int j = j0 + 8 * g, jb = j - (i >> 3) * a.rb;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e >= slots) v.h[e >> 2][e & 3] = 0.0f;
      if (wide && (jb < 0 || jb >= a.rb)) v.b = u32x4{0, 0, 0, 0};
      lo = slot_products<kF16>(v, lo);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) lo[e] *= a.s;
    return lo;
  };

  // A barrier that waits for this wave's LDS accesses, not for its copies in flight.
  auto meet = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  // The first batch's adapter, X, codes and the table, whose levels are picked in
  // front of all copies: a load behind them would wait for them.
  float lo = level(a.L, lane >> 2), hi = level(a.L, wave);
  asm volatile("" : "+v"(lo), "+v"(hi));
  Slots first;
  if (a.rb > 0 && wave < kGroups) first = load_slots(own, 0);
  __builtin_amdgcn_sched_barrier(0);
  // tokens 8 .. 15: waves 0 .. 7 in the ring's second slot, the others in its third
  unsigned char* const x0 = table + wave * kRegion;
  unsigned char* const x1 = (wave < 8 ? slot1 : slot2) + (wave & 7) * kRegion;
  copy_x(x0, 0, 0);
  if (kMany) copy_x(x1, 8, 0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < 8; ++j) xa[j] = u32x4{0, 0, 0, 0};
  stage(0, 0, 0);
  if (kMany) {
    wait_vmcnt<kOps>();  // X was copied in front of the codes
    __builtin_amdgcn_sched_barrier(0);
    read_x(x1, 8, 0);
    meet();  // every wave has read its part: the other slots may be filled
    stage(1, 0, 1);
    stage(2, 0, 2);
  } else {
    stage(1, 0, 1);
    stage(2, 0, 2);
    wait_vmcnt<3 * kOps>();
    __builtin_amdgcn_sched_barrier(0);
  }
  read_x(x0, 0, 0);
  f32x4 lora = f32x4{0.f, 0.f, 0.f, 0.f};
  if (a.rb > 0 && wave < kGroups) lora = adapter(first, own);
  meet();  // every wave has its X
  {
    // four threads an entry, eight of its copies each
    const u32x4 two = u32x4{__float_as_uint(lo), __float_as_uint(hi), __float_as_uint(lo), __float_as_uint(hi)};
#pragma unroll
    for (int c = 0; c < 4; ++c) *reinterpret_cast<u32x4*>(table + (tid >> 2) * 256 + (tid & 3) * 16 + c * 64) = two;
  }
  meet();
  const uint32_t copy = (lane & 31) * 8;
  auto look = [&](uint32_t c, u32x2(&pair)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      pair[e] = *reinterpret_cast<const u32x2*>(table + __builtin_amdgcn_perm(c, copy, 0x0C0C0400u | ((4u + e) << 8)));
  };
  const int codes = wave * kPart + i * 128;
  const int place = (2 * g) ^ ((i >> 1) & 7);  // of the lane's block, whose second half stands beside it, at place ^ 1

  f32x4 acc[kGroups];
  // A batch's groups from q0 on in one pass, whose first codes are on their way.
  auto multiply = [&](int q0, int pass) {
    const int have = live(pass) ? mine - q0 : 0;  // of the batch
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if (q >= have) break;
      const int slot = q % kAhead;
      __builtin_amdgcn_sched_barrier(0);
      // the first three groups are copied whether they exist or not
      if (q < kGroups - 2 && (q == 0 || q + 2 < have)) wait_vmcnt<2 * kOps>();
      else if (q < kGroups - 1 && (q <= 1 || q + 1 < have)) wait_vmcnt<kOps>();
      else wait_vmcnt<0>();
      __builtin_amdgcn_sched_barrier(0);
      const u32x4 c0 = ld16(ring[slot] + codes + 16 * place);
      const u32x4 c1 = ld16(ring[slot] + codes + 16 * (place ^ 1));
      const float s = kDQ ? dq_unit(sc[slot].code, a.w.dq) * sc[slot].value : sc[slot].value;
      if (q + kAhead < kGroups && q + kAhead < have) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the codes have left the slot
        __builtin_amdgcn_sched_barrier(0);
        stage(q0 + q + kAhead, pass, slot);
      }
      // the next eight weights' levels are read while these are scaled and multiplied
      u32x2 pair[2][4];
      look(c0[0], pair[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < 7) look(j < 3 ? c0[j + 1] : c1[j - 3], pair[(j + 1) & 1]);
        __builtin_amdgcn_sched_barrier(0);
        u32x4 wv;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u32x2 two = pair[j & 1][e];
          wv[e] = cvt_16x2<kF16>(__uint_as_float(two[0]) * s, __uint_as_float(two[1]) * s);
        }
        acc[q] = mma16<kF16>(xa[j], wv, acc[q]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_vmcnt<0>();  // copies of groups that do not exist
  };
  // A batch's sums and outputs; in one pass the next batch's first codes are on their
  // way before the outputs.
  auto finish = [&](int q0) {
    // acc[q][v]: token 4 g + v, row i of group q
    meet();  // the ring has been read
    const int lane = fresh_lane();
    auto sums = [&](int q) { return reinterpret_cast<f32x4*>(ring[q >> 1]) + (q & 1) * (kWaves * 64) + lane; };
#pragma unroll
    for (int q = 0; q < kGroups; ++q) sums(q)[wave * 64] = acc[q];
    meet();
    const bool owns = wave < kGroups && q0 + wave < mine;  // wave q sums group q
    f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
    if (owns) {
      const f32x4* red = reinterpret_cast<const f32x4*>(wave < 2 ? slot0 : wave < 4 ? slot1 : slot2) +
                         (wave & 1) * (kWaves * 64) + lane;
      sum = red[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += red[w * 64];
    }
    if (!kLong && q0 + kGroups < mine) {
      meet();  // the sums have been read
#pragma unroll
      for (int q = 0; q < kAhead; ++q) stage(q0 + kGroups + q, 0, q);
    }
    if (owns) {
      const int l = fresh_lane(), i = l & 15, g = l >> 4;
      const int out = group_of(q0 + wave) * 8 + (i & 7);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int token = 4 * g + v;
        const float up = __shfl_xor(sum[v], 8, 64);
        if (token >= a.M) continue;
        if (a.y != nullptr) a.y[static_cast<int64_t>(token) * N + out + (i >> 3) * half] = to16<kF16>(sum[v]);
        if (i < 8) a.p[static_cast<int64_t>(token) * half + out] = to16<kF16>(act_value<false>(sum[v], a.act) * up);
      }
    }
  };
  // Nothing is in flight: a further pass's X through the ring, then its first codes.
  auto restart = [&](int q0, int pass) {
    if (kLong) {
      for (int r0 = 0; r0 < a.M; r0 += 8) {
        __syncthreads();
        unsigned char* const at = (wave < 8 ? slot0 : slot1) + (wave & 7) * kRegion;
        copy_x(at, r0, pass);
        wait_vmcnt<0>();
        __builtin_amdgcn_sched_barrier(0);
        read_x(at, r0, pass);
      }
    }
    __syncthreads();  // the ring's codes, sums or X have been read
#pragma unroll
    for (int q = 0; q < kAhead; ++q) stage(q0 + q, pass, q);
  };
  auto begin = [&](f32x4 lora) {
#pragma unroll
    for (int q = 0; q < kGroups; ++q) acc[q] = q == wave ? lora : f32x4{0.f, 0.f, 0.f, 0.f};
  };

  // one copy of the loop's code, whose fetching from memory would cost as much as a batch
  for (int q0 = 0;;) {
    begin(lora);
    for (int pass = 0; pass < passes; ++pass) {
      if (kLong && q0 + pass > 0) restart(q0, pass);
      multiply(q0, pass);
    }
    finish(q0);
    q0 += kGroups;
    if (q0 >= mine) return;
    lora = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.rb > 0 && wave < kGroups) lora = adapter(load_slots(q0 + own, 0), q0 + own);
  }
}

// H = X A^T: a workgroup a row of A and up to 4 tokens, whose threads' sums of each
// token meet in LDS (16 wave sums by lane exchanges took 4 us of 7). 16 tokens, 32 rows of
// 4096: 3.4 us; 16 tokens a workgroup 4.8.
template <bool kF16>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  if constexpr (kF16) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, a), __builtin_bit_cast(h2, b), c, false);
  } else {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, a), __builtin_bit_cast(b2, b), c, false);
  }
}

constexpr int kHThreads = 512;

template <bool kF16, int kTokens>
__global__ __launch_bounds__(kHThreads) void gated_h_kernel(const uint16_t* x, int M, const uint16_t* a, int64_t K,
                                                            float* h) {
  x += blockIdx.y * kTokens * K;
  M -= blockIdx.y * kTokens;
  h += blockIdx.y * kTokens * gridDim.x;
  __shared__ float part[kTokens][kHThreads + 1];
  const int tid = threadIdx.x;
  float sum[kTokens];
#pragma unroll
  for (int t = 0; t < kTokens; ++t) sum[t] = 0.0f;
  const uint16_t* row = a + blockIdx.x * K;
  for (int64_t c = 8 * tid; c < K; c += 8 * kHThreads) {
    const u32x4 av = ld16(row + c);
    u32x4 xv[kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t) xv[t] = ld16(x + (t < M ? t : M - 1) * K + c);
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[t] = dot2<kF16>(av[e], xv[t][e], sum[t]);
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) part[t][tid] = sum[t];
  __syncthreads();
  const int token = tid / 32, at = tid % 32;
  if (token >= kTokens || token >= M) return;
  float v = 0.0f;
#pragma unroll
  for (int u = 0; u < kHThreads / 32; ++u) v += part[token][at + 32 * u];
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor(v, s, 64);
  if (at == 0) h[token * gridDim.x + blockIdx.x] = v;
}

}  // namespace

hipError_t launch_gated_h(const uint16_t* x, int64_t m, const uint16_t* a, int64_t k, int slots, float* h,
                          hipStream_t st, bool f16) {
  const int tokens = m <= 2 ? 2 : 4;
  auto kern = m <= 2 ? (f16 ? gated_h_kernel<true, 2> : gated_h_kernel<false, 2>)
                     : (f16 ? gated_h_kernel<true, 4> : gated_h_kernel<false, 4>);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(slots), static_cast<unsigned>((m + tokens - 1) / tokens)),
                     dim3(kHThreads), 0, st, x, static_cast<int>(m), a, k, h);
  return hipGetLastError();
}

hipError_t launch_gated_gemv(const PackedW& w, const uint16_t* x, int64_t m, const float* h, const uint16_t* b,
                             int rpart, float s, int act, uint16_t* y, uint16_t* p, hipStream_t st, bool f16) {
  Args a{w, x, 0, h, b, rpart, s, y, p, act, codebook_table(w.codebook)};
  const int64_t nrg = w.n / 16;
  const unsigned grid = static_cast<unsigned>(nrg < device_cus() ? nrg : device_cus());
  auto launch = [&](auto dq, auto half) {
    constexpr bool D = decltype(dq)::value, H = decltype(half)::value;
    auto kern = w.k > 4096 ? (a.M > 8 ? gated_gemv_kernel<D, H, true, true> : gated_gemv_kernel<D, H, true, false>)
                           : (a.M > 8 ? gated_gemv_kernel<D, H, false, true> : gated_gemv_kernel<D, H, false, false>);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(kThreads), 0, st, a);
  };
  for (int64_t t = 0; t < m; t += 16) {  // a launch for every 16 tokens
    a.M = static_cast<int>(m - t < 16 ? m - t : 16);
    a.x = x + t * w.k;
    a.h = h != nullptr ? h + t * 2 * rpart : nullptr;
    a.y = y != nullptr ? y + t * w.n : nullptr;
    a.p = p + t * (w.n / 2);
    if (f16) {
      if (w.dq) launch(std::true_type{}, std::true_type{});
      else launch(std::false_type{}, std::true_type{});
    } else {
      if (w.dq) launch(std::true_type{}, std::false_type{});
      else launch(std::false_type{}, std::false_type{});
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qlora
