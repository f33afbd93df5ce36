// The 8-bit product's choice of kernel and tile (int8_tiles.h), for CPU tests.
#include "int8_tiles.h"

// out: 1 for the kernel that streams the weight, the tile (-1 then, or where no
// tile fits), channels of a first launch (0: one launch), the tile of the second.
extern "C" void int8_choice(int64_t m, int64_t n, int64_t k, int64_t* out) {
  out[0] = qlora::decodes(m, n);
  out[1] = out[3] = -1;
  out[2] = 0;
  if (out[0]) return;
  const qlora::Pick one = qlora::pick_shape(m, n, k);
  out[1] = one.shape;
  out[2] = qlora::full_rounds(m, n, k, one);
  if (out[2] > 0) out[3] = qlora::pick_shape(m, n - out[2], k).shape;
}

// out: tokens, channels, groups along the contraction, parts of the ring.
extern "C" int int8_tile(int i, int64_t* out) {
  if (i < 0 || i >= qlora::kNumShapes) return 0;
  const qlora::Shape s = qlora::kShapes[i];
  out[0] = s.bm;
  out[1] = s.bn;
  out[2] = s.groups;
  out[3] = s.parts;
  return 1;
}
