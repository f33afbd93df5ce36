// Which kernel and tile an 8-bit product runs on: host arithmetic alone, so
// that tests can ask it without a GPU.
#pragma once

#include <stdint.h>

namespace qlora {

// At most these tokens and channels: the kernel that streams the weight (both
// sides' times stand beside it, in int8_gemm.hip).
constexpr int kDecodeTokens = 16;
constexpr int kDecodeMaxN = 8191;
inline bool decodes(int64_t m, int64_t n) { return m <= kDecodeTokens && n <= kDecodeMaxN; }

// The tile for a call: the one with the least kLaunch + rounds * (round + units *
// unit) microseconds, where rounds counts turns of the 256 CUs, units steps of
// 128 codes, `round` a tile's start and its outputs. Fitted to measured times
// (graph replays, bf16 out). Over 48 sizes drawn from 1 .. 4096 tokens, 64 ..
// 22016 channels and 64 .. 11008 codes its choice takes 1.4% longer on average
// than the best tile for each. Some of the times behind it (m x n x k, us):
//   4096 x 8192 x 8192:  256 x 256 206, 128 x 256 238, 128 x 128 317
//   2048 x 4096 x 11008: 128 x 256 76, 128 x 128 92, 256 x 256 102
//   2048 x 11008 x 4096: 128 x 256 90, 256 x 256 104, 128 x 128 119
//   512 x 4096 x 4096:   64 x 128 14.8, 64 x 64 17.6, 128 x 128 19.0
//   128 x 4096 x 4096:   32 x 64 8.6, 64 x 64 10.8, 64 x 128 12.5
//   64 x 11008 x 4096:   64 x 64 11.3, 64 x 128 13.5, 32 x 64 15.9
//   32 x 4096 x 11008:   16 x 64 14.4, 32 x 64 17.1
//   745 x 21599 x 147:   256 x 256 22, 128 x 256 24, 64 x 64 34, 16 x 64 96
struct Shape {
  int bm, bn;     // tokens, channels
  int wm, wn;     // waves along the two
  int groups;     // of wm x wn waves, which share the contraction
  int parts;      // of a group's LDS ring
  double round, unit;
  constexpr int threads() const { return 64 * wm * wn * groups; }
};
constexpr Shape kShapes[] = {
    {256, 256, 2, 4, 1, 5, 12, 1.4}, {128, 256, 2, 4, 1, 6, 8, 0.78}, {128, 128, 2, 2, 1, 8, 4.5, 0.5},
    {64, 128, 2, 2, 1, 8, 3, 0.34},  {64, 64, 4, 1, 1, 8, 1.4, 0.22}, {32, 64, 2, 1, 2, 8, 2.2, 0.14},
    {16, 64, 1, 1, 2, 8, 1.2, 0.13}};
constexpr int kNumShapes = sizeof(kShapes) / sizeof(kShapes[0]);
constexpr double kLaunch = 2;

inline int64_t tiles_of(const Shape& s, int64_t m, int64_t n) { return ((m + s.bm - 1) / s.bm) * ((n + s.bn - 1) / s.bn); }

inline double cost(const Shape& s, int64_t tiles, int64_t k) {
  return kLaunch + static_cast<double>((tiles + 255) / 256) * (s.round + static_cast<double>((k + 127) / 128) * s.unit);
}

struct Pick {
  int shape;  // into kShapes; -1: no tile's grid stays below 2^32 work items
  double us;
};
inline Pick pick_shape(int64_t m, int64_t n, int64_t k) {
  Pick best{-1, 0};
  for (int i = 0; i < kNumShapes; ++i) {
    const int64_t tiles = tiles_of(kShapes[i], m, n);
    if (tiles >= (INT64_C(1) << 32) / kShapes[i].threads()) continue;
    const double us = cost(kShapes[i], tiles, k);
    if (best.shape < 0 || us < best.us) best = Pick{i, us};
  }
  return best;
}

// Channels of a first launch in 256 x 256 tiles whose rounds are full, where
// these and a second launch for the other channels cost less than one launch;
// 0 where they do not. 4096 x 22016 x 8192 has 1376 tiles, 5.4 rounds: 574 us
// in one launch, 551 us as five full rounds and 192 tiles of 128 x 256.
inline int64_t full_rounds(int64_t m, int64_t n, int64_t k, const Pick& one) {
  const int64_t tiles_m = (m + 255) / 256, tiles = tiles_of(kShapes[0], m, n);
  if (one.shape != 0 || tiles_m > 256 || tiles % 256 == 0) return 0;
  const int64_t cols = tiles / 256 * 256 / tiles_m * 256;
  if (cols < 256 || cols >= n) return 0;
  return cost(kShapes[0], tiles_of(kShapes[0], m, cols), k) + pick_shape(m, n - cols, k).us < one.us ? cols : 0;
}

}  // namespace qlora
