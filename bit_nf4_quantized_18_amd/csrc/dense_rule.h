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
//   1040 x 1088, 16 slots  16.5 / 23.3, 31 / 39; 64 slots 19.0 / 27.3, 43 / 55
//   2048 x 2048, 16 slots  21.0 / 24.1, 43 / 48; 64 slots 23.0 / 29.2, 57 / 68
//   4096 x 4096, 16 slots  41.4 / 39.5, 94 / 96; 64 slots 44.9 / 44.1, 118 / 121
//   6656 x 4544, 16 slots  57.2 / 47.3, 167 / 161; 64 slots 61.0 / 50.8, 204 / 195
constexpr int64_t kDenseNarrow = 4096;
inline bool dense_narrow(int64_t n) { return n <= kDenseNarrow; }

// m tokens, `out` weight rows along the outputs (of the stored weight or of its
// transpose), `con` elements of contraction. A launch has under 2^32 threads, up to
// 512 a token for H or dH.
inline bool dense_fits(int64_t m, int64_t out, int64_t con) {
  return con <= kDenseMaxK && m < (INT64_C(1) << 22) && pick_shape(m, out, 2 * con).shape >= 0;
}

// The two sides' microseconds, fitted to 114 measured calls (17 .. 4096 tokens, 0.5 M
// .. 360 M weights, forward and backward, rank 16), where the smaller estimate names the
// slower side by more than 2% twice (3% and 4%). Fused: rounds of the 256 CUs over 256 x
// 128 tiles, in steps of 64, and H or dH in launches of their own. Dense: 2.5 bytes a
// weight to restore it, then the tiles of the 8-bit product, whose units of 128 bytes
// take about as long, or reading 2 bytes a weight.
// Some of the calls, fused / dense, us:
//   tokens                            64           333          2048         4096
//   forward 22016 x 4096          65 / 71     123 / 121     392 / 350    745 / 647
//   forward 44032 x 8192        221 / 350                 1389 / 1279
//   forward 2560 x 5120           75 / 41       79 / 42       81 / 78    158 / 121
//   forward 5120 x 1088           30 / 18       31 / 23       55 / 43      83 / 73
//   tokens                            64           256          1024         4096
//   backward 22016 x 4096       278 / 108     282 / 136     294 / 258    735 / 650
//   backward 4096 x 11008         72 / 53       74 / 66     141 / 121    409 / 347
//   backward 8192 x 22016       119 / 222     123 / 253     382 / 462
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
