// Host driver for the 8-bit and gradient entry points. api.cpp is built with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host side and linked
// with the library's kernel objects. Argument checks, list handling (lengths,
// overlaps, workspace sizes) and valid calls on host buffers, whose first
// launch fails because no GPU is visible; that part is skipped if one is.
// Prints "abi_int8_sanitize: all checks passed" and exits 0, or names every
// failed check and exits 1.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
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
  std::vector<float> pool(1 << 16);
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(pool.data()) + 255) & ~uintptr_t{255});
  int8_t* codes = reinterpret_cast<int8_t*>(base);
  float* scale = reinterpret_cast<float*>(base + 8192);
  void* x = base + 16384;
  void* y = base + 65536;
  float* norm = reinterpret_cast<float*>(base + 4096);

  // sizes at the ends of their ranges
  const int64_t big = INT64_MAX;
  CHECK_EQ(qlora_int8_quantize(x, QLORA_F32, big, 64, codes, 64, scale, nullptr), QLORA_ERR_SHAPE);
  CHECK_EQ(qlora_int8_quantize(x, QLORA_F32, 1, big, codes, 64, scale, nullptr), QLORA_ERR_SHAPE);
  CHECK_EQ(qlora_int8_quantize(x, QLORA_F32, 1, 64, codes, big, scale, nullptr), QLORA_ERR_SHAPE);
  CHECK_EQ(qlora_int8_dequantize(codes, INT64_MIN, scale, 1, 64, QLORA_F32, y, nullptr), QLORA_ERR_SHAPE);
  CHECK_EQ(qlora_rmsnorm_int8(x, nullptr, x, QLORA_BF16, QLORA_BF16, INT64_MIN, 64, 0.0f, nullptr, codes, 64, scale,
                              nullptr), QLORA_ERR_SHAPE);
  CHECK_EQ(qlora_rmsnorm_int8(x, nullptr, x, QLORA_BF16, QLORA_BF16, 1, 64, HUGE_VALF, nullptr, codes, 64, scale,
                              nullptr), QLORA_ERR_UNSUPPORTED);
  for (int64_t m : {INT64_C(1), INT64_C(17), INT64_C(2147483647), big})
    for (int64_t n : {INT64_C(1), INT64_C(4194304), big, INT64_MIN})
      for (int64_t k : {INT64_C(63), INT64_C(131072), big, INT64_MIN})
        CHECK_EQ(qlora_int8_linear_fwd(codes, scale, n, k, codes, scale, m, QLORA_BF16, y, nullptr), QLORA_ERR_SHAPE);
  CHECK_EQ(qlora_int8_linear_fwd(codes, scale, 1, 64, codes, scale, 2147483647, QLORA_BF16, y, nullptr),
           QLORA_ERR_SHAPE);  // more tiles than a launch takes

  // lists: none, empty tensors, many, lengths whose sum leaves 64 bits
  CHECK_EQ(qlora_grad_workspace_bytes(nullptr, 0) == 0, 1);
  std::vector<int64_t> len(1000);
  std::vector<void*> at(1000);
  for (int i = 0; i < 1000; ++i) {
    len[i] = i % 7 == 0 ? 0 : i % 5 + 1;
    at[i] = base + 16384 + 64 * ((i * 617) % 1000);  // apart, in no order
  }
  const size_t need = qlora_grad_workspace_bytes(len.data(), 1000);
  CHECK_EQ(need > 0 && need < 131072, 1);
  std::vector<char> wsbuf(need + 256);
  void* ws = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(wsbuf.data()) + 255) & ~uintptr_t{255});
  CHECK_EQ(qlora_grad_clip(at.data(), len.data(), 1000, QLORA_F32, 1.0f, nullptr, norm, ws, need - 1, nullptr),
           QLORA_ERR_WORKSPACE);
  void* kept = at[999];
  at[999] = static_cast<char*>(at[1]) + 4;  // inside another tensor
  CHECK_EQ(qlora_grad_clip(at.data(), len.data(), 1000, QLORA_F32, 1.0f, nullptr, norm, ws, need, nullptr),
           QLORA_ERR_UNSUPPORTED);
  at[999] = kept;
  CHECK_EQ(qlora_grad_clip(at.data(), len.data(), 1000, QLORA_F32, 1.0f, at[500], norm, ws, need, nullptr),
           QLORA_ERR_UNSUPPORTED);
  int64_t huge[3] = {big, big, big};
  CHECK_EQ(qlora_grad_workspace_bytes(huge, 3), 0);
  CHECK_EQ(qlora_grad_clip(at.data(), huge, 3, QLORA_F32, 1.0f, nullptr, norm, ws, need, nullptr), QLORA_ERR_SHAPE);
  int64_t most[1] = {INT64_C(1) << 40};
  CHECK_EQ(qlora_grad_workspace_bytes(most, 1) > 0, 1);

  int devices = 0;
  if (hipGetDeviceCount(&devices) != hipSuccess || devices == 0) {
    (void)hipGetLastError();
    CHECK_EQ(qlora_int8_quantize(x, QLORA_F32, 2, 100, codes, 128, scale, nullptr), QLORA_ERR_HIP);
    CHECK_EQ(qlora_int8_dequantize(codes, 128, scale, 2, 100, QLORA_F16, y, nullptr), QLORA_ERR_HIP);
    CHECK_EQ(qlora_rmsnorm_int8(x, x, x, QLORA_BF16, QLORA_F32, 2, 100, 1e-6f, y, codes, 128, scale, nullptr),
             QLORA_ERR_HIP);
    for (int64_t m : {1, 40, 300})
      CHECK_EQ(qlora_int8_linear_fwd(codes, scale, 8, 64, codes, scale, m, QLORA_F32, y, nullptr), QLORA_ERR_HIP);
    CHECK_EQ(qlora_int8_linear_fwd(codes, scale, 53248, 1856, codes, scale, 1000, QLORA_F32, y, nullptr), QLORA_ERR_HIP);
    CHECK_EQ(qlora_grad_clip(at.data(), len.data(), 1000, QLORA_F32, 1.0f, nullptr, norm, ws, need, nullptr),
             QLORA_ERR_HIP);
    CHECK_EQ(qlora_grad_norm(at.data(), len.data(), 1000, QLORA_BF16, norm, ws, need, nullptr), QLORA_ERR_HIP);
    CHECK_EQ(qlora_grad_norm(nullptr, nullptr, 0, QLORA_F32, norm, nullptr, 0, nullptr), QLORA_ERR_HIP);
  } else {
    std::printf("a GPU is visible: launches skipped\n");
  }
  if (g_failures == 0) std::printf("abi_int8_sanitize: all checks passed\n");
  return g_failures == 0 ? 0 : 1;
}
