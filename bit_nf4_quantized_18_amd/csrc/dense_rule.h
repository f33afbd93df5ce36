// Whether a product over m tokens restores its NF4 weight once, into the workspace,
// and multiplies it from there (dense_gemm.hip), or restores it as it multiplies
// (gemm_kernels.hip): host arithmetic alone, so that tests can ask it without a GPU.
#pragma once

#include "int8_tiles.h"

namespace qlora {

// Longest contraction of the dense kernels: 32-bit offsets in a tile of 256 rows.
constexpr int64_t kDenseMaxK = 65536;

// m tokens, `out` weight rows along the outputs (of the stored weight or of its
// transpose), `con` elements of contraction.
inline bool dense_fits(int64_t m, int64_t out, int64_t con) {
  return con <= kDenseMaxK && pick_shape(m, out, 2 * con).shape >= 0;
}

// The two sides' microseconds, fitted to 114 measured calls (17 .. 4096 tokens, 0.5 M
// .. 360 M weights, forward and backward), where the smaller estimate names the slower
// side by more than 2% once. Fused: rounds of the 256 CUs over 256 x 128 tiles, in steps
// of 64. Dense: 2.5 bytes a weight to restore it, then the tiles of the 8-bit product,
// whose units of 128 bytes take about as long, or reading 2 bytes a weight.
// Some of the calls, fused / dense, us:
//   tokens                            64           333          2048         4096
//   forward 22016 x 4096          65 / 96     123 / 147     382 / 360    712 / 635
//   forward 2560 x 5120           75 / 47       79 / 44       81 / 95    159 / 133
//   forward 5120 x 1088           31 / 25       32 / 29       55 / 51      78 / 85
//   tokens                            64           256          1024         4096
//   backward 22016 x 4096       278 / 129     282 / 155     296 / 280    711 / 627
//   backward 4096 x 11008         73 / 57       74 / 71     141 / 126    402 / 334
//   backward 8192 x 22016       119 / 227     123 / 261     370 / 468
inline bool dense_pays(int64_t m, int64_t out, int64_t con) {
  if (!dense_fits(m, out, con)) return false;
  const int64_t tiles = ((m + 255) / 256) * ((out + 127) / 128);
  const double fused = static_cast<double>((tiles + 255) / 256) * (6 + 0.9 * static_cast<double>((con + 63) / 64));
  const double weights = static_cast<double>(out) * static_cast<double>(con);
  const double product = pick_shape(m, out, 2 * con).us, read = weights * 2 / 3.0e6;
  return weights * 2.5 / 5.0e6 + (product > read ? product : read) < fused;
}

}  // namespace qlora
