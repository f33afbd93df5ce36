// Whether a product over m tokens restores its NF4 weight once, into the workspace,
// and multiplies it from there (dense_gemm.hip), or restores it as it multiplies
// (gemm_kernels.hip): host arithmetic alone, so that tests can ask it without a GPU.
#pragma once

#include "int8_tiles.h"

namespace qlora {

// Longest contraction of the dense kernels: 32-bit offsets in a tile of 256 rows.
constexpr int64_t kDenseMaxK = 65536;

// Whether dH = s dY B over n weight rows is formed beside the restoring, 16 tokens and
// 16 slots a workgroup whose lanes read B in strided loads, or behind it from B^T. Whole
// calls, us, beside / behind, 17 and 2048 tokens:
//   1040 x 1088, 16 slots  18.3 / 23.6, 35 / 41; 64 slots 21.0 / 29.1, 44 / 56
//   2048 x 2048, 16 slots  22.6 / 25.3, 45 / 50; 64 slots 24.6 / 30.9, 55 / 63
//   4096 x 4096, 16 slots  42.4 / 40.8, 94 / 95; 64 slots 46.5 / 45.8, 111 / 114
//   6656 x 4544, 16 slots  59.2 / 48.3, 170 / 164; 64 slots 62.8 / 52.6, 198 / 189
constexpr int64_t kDenseNarrow = 4096;
inline bool dense_narrow(int64_t n) { return n <= kDenseNarrow; }

// m tokens, `out` weight rows along the outputs (of the stored weight or of its
// transpose), `con` elements of contraction. A launch has under 2^32 threads, up to
// 512 a token for H or dH.
inline bool dense_fits(int64_t m, int64_t out, int64_t con) {
  return con <= kDenseMaxK && m < (INT64_C(1) << 22) && pick_shape(m, out, 2 * con).shape >= 0;
}

// The two sides' microseconds, to choose by and no more: fitted to 114 measured calls (17
// .. 4096 tokens, 0.5 M .. 360 M weights, forward and backward, rank 16), where the
// smaller estimate names the slower side by more than 2% twice (3% and 4%). Fused: rounds
// of the 256 CUs over 256 x 128 tiles, in steps of 64, and H or dH in launches of their
// own. Dense: 2.5 bytes a weight to restore it, then the tiles of the 8-bit product, whose
// units of 128 bytes take about as long, or reading 2 bytes a weight. Few tokens of a
// large weight are estimated high on that side (64 x 22016 x 4096: 105 us, 71 measured: the
// restored weight is read back faster than counted), where the fused side still is the
// faster one. A side that gets faster needs the fit again.
// Some of the calls, fused / dense, us:
//   tokens                            64           333          2048         4096
//   forward 22016 x 4096          67 / 71     125 / 122     396 / 346    739 / 635
//   forward 44032 x 8192        222 / 340     345 / 526   1366 / 1285  2733 / 2327
//   forward 2560 x 5120           75 / 38       81 / 40       83 / 79    161 / 129
//   forward 5120 x 1088           31 / 19       33 / 22       59 / 45      87 / 80
//   tokens                            64           256          1024         4096
//   backward 22016 x 4096       282 / 113     287 / 142     295 / 251    711 / 637
//   backward 4096 x 11008         74 / 54       76 / 68     141 / 121    412 / 350
//   backward 8192 x 22016       121 / 221     127 / 254     378 / 463  1373 / 1209
inline double fused_us(int64_t m, int64_t out, int64_t con) {
  const int64_t tiles = ((m + 255) / 256) * ((out + 127) / 128);
  return 6 + static_cast<double>((tiles + 255) / 256) * (6 + 0.9 * static_cast<double>((con + 63) / 64));
}

inline double dense_us(int64_t m, int64_t out, int64_t con) {
  const double weights = static_cast<double>(out) * static_cast<double>(con);
  const double product = pick_shape(m, out, 2 * con).us, read = weights * 2 / 3.0e6;
  return weights * 2.5 / 5.0e6 + (product > read ? product : read);
}

inline bool dense_pays(int64_t m, int64_t out, int64_t con) {
  return dense_fits(m, out, con) && dense_us(m, out, con) < fused_us(m, out, con);
}

// Whether a gated block of n weight rows takes its tokens 16 at a time through the
// decode kernel, which reads the packed weight again for each 16: always up to 16, and
// up to 32 where two launches, about 17 us and 0.3 a million weights with H, cost less
// than the better product above. 32 tokens, two launches / the product, us:
//   5120 x 1088   19 / 15      11264 x 2048  23 / 31      10240 x 2560  24 / 35
//   16384 x 4096  33 / 63      22016 x 4096  39 / 63      28672 x 4096  51 / 66
//   27648 x 5120  72 / 76      44032 x 8192  138 / 218
// (2560 x 5120, 31 / 40, is left to the product), and 33 tokens in three: 22016 x 4096
// 61 / 62, 28672 x 4096  77 / 66.
inline bool gated_decodes(int64_t m, int64_t n, int64_t k) {
  if (m <= 16) return true;
  if (m > 32) return false;
  const double fused = fused_us(m, n, k), dense = dense_fits(m, n, k) ? dense_us(m, n, k) : fused;
  return 17 + 0.3e-6 * static_cast<double>(n) * static_cast<double>(k) < (dense < fused ? dense : fused);
}

}  // namespace qlora
