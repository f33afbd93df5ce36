// Host driver for the gated-block calls and the backward calls from 8-bit rows. api.cpp
// is built with AddressSanitizer and UndefinedBehaviorSanitizer on the host side and
// linked with the library's kernel objects. Sizes at the ends of their ranges, workspace
// sizes over the whole range, overlaps, and valid calls, whose first launch fails because
// no GPU is visible; that part is skipped if one is. Prints "abi_gated_sanitize: all
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
  const int64_t big = INT64_MAX, least = INT64_MIN;

  // workspace sizes: 0 for bad sizes, no overflow for good ones
  const int64_t ms[] = {least, -1, 0, 1, 16, 17, 32, 33, 300, 1 << 20, INT64_C(1) << 31, (INT64_C(1) << 31) + 1, big};
  const int64_t dims[] = {least, 0, 16, 64, 512, 22016, 1 << 22, (1 << 22) + 1, big};
  for (int64_t m : ms)
    for (int64_t n : dims)
      for (int64_t k : dims)
        for (int r : {INT32_MIN, -1, 0, 1, 16, 64, 65, INT32_MAX / 2}) {
          const bool sizes = m > 0 && m <= INT64_C(1) << 31 && n > 0 && n <= 1 << 22 && k > 0 && k <= 1 << 22;
          const bool none = !sizes || r < 0 || r > 64 || (r == 0 && m <= 16);
          if (none) CHECK_EQ(qlora_linear_gated_workspace_bytes(m, n, k, r), 0);
          else if (r > 0) CHECK_EQ(qlora_linear_gated_workspace_bytes(m, n, k, r) > 0, 1);
          for (int g : {INT32_MIN, 0, 1, 2, 4, 5}) {
            const bool bad = !sizes || g < 1 || g > 4 || r < 0 || int64_t{g} * r > 128;
            if (bad && r <= 64) CHECK_EQ(qlora_linear_x8_workspace_bytes(m, n, k, g, r), 0);
            else if (!bad && r > 0) CHECK_EQ(qlora_linear_x8_workspace_bytes(m, n, k, g, r) > 0, 1);
          }
        }

  std::vector<char> pool(1 << 22);
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(pool.data()) + 255) & ~uintptr_t{255});
  auto at = [&](int i) { return base + (i << 17); };
  auto u16 = [&](int i) { return reinterpret_cast<uint16_t*>(at(i)); };
  auto f32 = [&](int i) { return reinterpret_cast<float*>(at(i)); };
  auto i8 = [&](int i) { return reinterpret_cast<int8_t*>(at(i)); };

  // elementwise and 8-bit calls at the ends of their ranges
  for (int64_t m : {least, int64_t{-1}, INT64_C(1) << 30, big}) {
    CHECK_EQ(qlora_gated_fwd(at(0), QLORA_BF16, m, 64, 0, at(1), nullptr), QLORA_ERR_SHAPE);
    CHECK_EQ(qlora_gated_bwd_x8(i8(0), 64, f32(1), at(2), QLORA_F32, m, 64, 0, at(3), nullptr), QLORA_ERR_SHAPE);
  }
  for (int64_t n : {least, int64_t{0}, (INT64_C(1) << 22) + 1, big}) {
    CHECK_EQ(qlora_gated_bwd(at(0), at(1), QLORA_F16, 1, n, 1, at(2), nullptr), QLORA_ERR_SHAPE);
    CHECK_EQ(qlora_gated_fwd_x8(i8(0), big, f32(1), QLORA_F32, 1, n, 0, at(3), nullptr), QLORA_ERR_SHAPE);
    CHECK_EQ(qlora_int8_linear_fwd_gated(i8(0), f32(1), n, 64, i8(2), f32(3), 1, 0, QLORA_BF16, at(4), nullptr),
             QLORA_ERR_SHAPE);
  }
  CHECK_EQ(qlora_int8_linear_fwd_gated(i8(0), f32(1), 1 << 21, 64, i8(2), f32(3), INT64_C(1) << 31, 0, QLORA_BF16, at(4),
                                       nullptr), QLORA_ERR_SHAPE);

  // a weight of 512 x 64: argument errors, then valid calls
  const qlora_nf4_weight w{512, 64, reinterpret_cast<uint8_t*>(at(0)), reinterpret_cast<uint8_t*>(at(1)), f32(2), nullptr, 1, 0};
  const size_t ws = qlora_linear_gated_workspace_bytes(20, 512, 64, 16), ws8 = qlora_linear_x8_workspace_bytes(20, 512, 64, 2, 16);
  const int64_t parts[] = {256, 256};
  auto block = [&](int64_t m, int act, size_t bytes, uint16_t* p) {
    return qlora_linear_fwd_gated(&w, u16(3), m, u16(4), u16(5), 16, 32.0f, act, u16(6), p, f32(8), at(9), bytes, nullptr);
  };
  auto back = [&](int64_t ld, size_t bytes, uint16_t* dx) {
    return qlora_linear_bwd_grouped_x8(&w, 2, parts, i8(10), ld, f32(11), u16(12), 20, u16(4), u16(5), 16, 32.0f, f32(13),
                                       dx, f32(15), f32(16), at(17), bytes, nullptr);
  };
  CHECK_EQ(block(least, 0, ws, u16(7)), QLORA_ERR_SHAPE);
  CHECK_EQ(block(20, 7, ws, u16(7)), QLORA_ERR_UNSUPPORTED);
  CHECK_EQ(block(20, 0, 16, u16(7)), QLORA_ERR_WORKSPACE);
  CHECK_EQ(block(20, 0, ws, u16(3)), QLORA_ERR_UNSUPPORTED);
  CHECK_EQ(back(least, ws8, u16(14)), QLORA_ERR_SHAPE);
  CHECK_EQ(back(big - 63, ws8, u16(14)), QLORA_ERR_SHAPE);
  CHECK_EQ(back(64, 16, u16(14)), QLORA_ERR_WORKSPACE);
  CHECK_EQ(back(64, ws8, u16(12)), QLORA_ERR_UNSUPPORTED);
  int devices = 0;
  if (hipGetDeviceCount(&devices) != hipSuccess || devices == 0) {
    for (int64_t m : {1, 9, 20}) CHECK_EQ(block(m, 1, ws, u16(7)), QLORA_ERR_HIP);
    CHECK_EQ(back(64, ws8, u16(14)), QLORA_ERR_HIP);
    CHECK_EQ(qlora_gated_bwd(at(0), at(1), QLORA_BF16, 4, 100, 0, at(0), nullptr), QLORA_ERR_HIP);
    CHECK_EQ(qlora_int8_linear_fwd_gated(i8(0), f32(1), 100, 64, i8(2), f32(3), 4, 0, QLORA_F32, at(4), nullptr), QLORA_ERR_HIP);
  }
  if (g_failures == 0) std::printf("abi_gated_sanitize: all checks passed\n");
  return g_failures == 0 ? 0 : 1;
}
