// Host driver for arguments far outside their ranges in the grouped, gated-block and
// 8-bit backward calls: api.cpp is built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host side and linked with the library's kernel
// objects, with every device hidden. Prints "abi_ranges_sanitize: all
// checks passed" and exits 0, or names every failed check and exits 1.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <vector>

#include "qlora_nf4.h"

static int g_failures = 0;

#define CHECK_EQ(expr, want)                                                                            \
  do {                                                                                                  \
    const long long got_ = static_cast<long long>(expr);                                                \
    const long long want_ = static_cast<long long>(want);                                               \
    if (got_ != want_) {                                                                                \
      std::fprintf(stderr, "FAILED line %d: %s = %lld, expected %lld\n", __LINE__, #expr, got_, want_); \
      ++g_failures;                                                                                     \
    }                                                                                                   \
  } while (0)

int main() {
  std::vector<char> pool(1 << 22);
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(pool.data()) + 255) & ~uintptr_t{255});
  auto at = [&](int i) { return base + (i << 17); };
  auto u16 = [&](int i) { return reinterpret_cast<uint16_t*>(at(i)); };
  auto f32 = [&](int i) { return reinterpret_cast<float*>(at(i)); };
  auto i8 = [&](int i) { return reinterpret_cast<int8_t*>(at(i)); };
  const qlora_nf4_weight w{1024, 64, reinterpret_cast<uint8_t*>(at(0)), reinterpret_cast<uint8_t*>(at(1)), f32(2), nullptr, 1, 0};
  const size_t many = SIZE_MAX;

  // ranks whose products with the number of parts leave an int
  for (int r : {129, INT32_MAX / 4 + 1, INT32_MAX / 3 + 1, INT32_MAX / 2, (1 << 30), (1 << 30) + 16, INT32_MAX - 15, INT32_MAX}) {
    for (int64_t m : {1, 300}) CHECK_EQ(qlora_linear_gated_workspace_bytes(m, 1024, 64, r), 0);
    CHECK_EQ(qlora_linear_fwd_gated(&w, u16(3), 20, u16(4), u16(5), r, 32.0f, 0, u16(6), u16(7), f32(8), at(9), many, nullptr),
             QLORA_ERR_UNSUPPORTED);
    for (int g : {1, 2, 3, 4}) {
      CHECK_EQ(qlora_linear_x8_workspace_bytes(300, 1024, 64, g, r), 0);
      CHECK_EQ(qlora_linear_grouped_workspace_bytes(300, 1024, 64, g, r), 0);
    }
    const int64_t parts[] = {256, 256, 256, 256};
    for (uint16_t* dx : {static_cast<uint16_t*>(nullptr), u16(14)}) {
      CHECK_EQ(qlora_linear_bwd_grouped_x8(&w, 4, parts, i8(10), 64, f32(11), u16(12), 20, u16(4), u16(5), r, 32.0f, f32(13),
                                           dx, f32(15), f32(16), at(17), many, nullptr), QLORA_ERR_UNSUPPORTED);
      CHECK_EQ(qlora_linear_bwd_grouped(&w, 4, parts, u16(10), u16(12), 20, u16(4), u16(5), r, 32.0f, f32(13), dx, f32(15),
                                        f32(16), at(17), many, nullptr), QLORA_ERR_UNSUPPORTED);
    }
    CHECK_EQ(qlora_linear_fwd_grouped(&w, 4, parts, u16(3), 20, u16(4), u16(5), r, 32.0f, u16(6), f32(8), at(9), many, nullptr),
             QLORA_ERR_UNSUPPORTED);
  }

  // row lengths of inputs that are not read (no adapter) are not multiplied either; the
  // call itself is fine and ends at its first launch, no device being visible
  for (int64_t ld : {INT64_MIN, int64_t{-64}, int64_t{0}, INT64_MAX - 63, INT64_MAX})
    for (int8_t* x : {static_cast<int8_t*>(nullptr), i8(10)}) {
      CHECK_EQ(qlora_linear_bwd_x8(&w, x, ld, f32(11), u16(12), 20, nullptr, nullptr, 0, 32.0f, nullptr, u16(14), nullptr,
                                   nullptr, at(17), many, nullptr), QLORA_ERR_HIP);
      CHECK_EQ(qlora_linear_bwd_x8(&w, x, ld, f32(11), u16(12), 20, u16(4), u16(5), 16, 32.0f, f32(13), u16(14), f32(15),
                                   f32(16), at(17), many, nullptr), x == nullptr ? QLORA_ERR_NULL : QLORA_ERR_SHAPE);
    }
  if (g_failures == 0) std::printf("abi_ranges_sanitize: all checks passed\n");
  return g_failures == 0 ? 0 : 1;
}
