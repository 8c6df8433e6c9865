// Drives the entry points of serve_abi.cpp through accepted and rejected
// arguments against the stand-in launchers: the status of each call, one
// launch for an accepted call that has work, none otherwise.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "gptq.h"

extern int g_launches;

namespace {
int g_fails = 0, g_checks = 0;
void check(int got, int want, int launched, int want_launched, const char* what, int line) {
  ++g_checks;
  if (got != want || launched != want_launched) {
    std::printf("FAIL line %d: %s returned %d (want %d), launched %d (want %d)\n", line, what, got,
                want, launched, want_launched);
    ++g_fails;
  }
}
#define EXPECT(call, want, launches)                                     \
  do {                                                                   \
    const int before = g_launches;                                       \
    const int got = (call);                                              \
    check(got, (want), g_launches - before, (launches), #call, __LINE__); \
  } while (0)
}  // namespace

int main() {
  alignas(256) static unsigned char buf[4096];
  void* p = buf;
  auto* q = (uint32_t*)p;
  auto* h = (uint16_t*)p;
  auto* f = (float*)p;
  auto* x8 = (int8_t*)p;
  const int64_t big = std::numeric_limits<int64_t>::max();
  // a few tokens
  EXPECT(gptq_w4a16_matvec(p, 1, 256, q, h, h, 8, 256, 128, 0, f, nullptr, 0, nullptr), GPTQ_OK, 1);
  EXPECT(gptq_w4a16_matvec(p, 64, 256, q, h, nullptr, 8, 256, -1, 1, f, p, 2048, nullptr), GPTQ_OK, 1);
  EXPECT(gptq_w4a16_matvec(p, 64, 256, q, h, nullptr, 8, 256, -1, 1, f, p, 2047, nullptr), GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a16_matvec(p, 64, 256, q, h, nullptr, 8, 256, -1, 1, f, nullptr, 2048, nullptr), GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a16_matvec(p, 64, 256, q, h, nullptr, 8, 256, -1, 1, f, buf + 128, 2048, nullptr), GPTQ_EINVAL, 0);
  EXPECT((int)gptq_w4a16_matvec_workspace(64, 8, 256, 32), 2048, 0);
  EXPECT((int)gptq_w4a16_matvec_workspace(65, 8, 256, 32), 0, 0);
  EXPECT((int)gptq_w4a16_matvec_workspace(64, 8, 250, 32), 0, 0);
  EXPECT(gptq_w4a16_matvec(p, 0, 256, q, h, h, 8, 256, 128, 0, f, nullptr, 0, nullptr), GPTQ_OK, 0);
  EXPECT(gptq_w4a16_matvec(p, 65, 256, q, h, h, 8, 256, 128, 0, f, nullptr, 0, nullptr), GPTQ_EUNSUPPORTED, 0);
  EXPECT(gptq_w4a16_matvec(p, 1, 256, q, h, nullptr, 8, 256, 128, 0, f, nullptr, 0, nullptr), GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a16_matvec(p, 1, big, q, h, h, 8, 256, 128, 0, f, nullptr, 0, nullptr), GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a16_matvec(p, big, 256, q, h, h, 8, 256, 128, 0, f, nullptr, 0, nullptr), GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a16_matvec(p, 1, 256, q, h, h, big, 256, 128, 0, f, nullptr, 0, nullptr), GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a16_matvec(p, 1, 256, q, h, h, 8, big, 128, 0, f, nullptr, 0, nullptr), GPTQ_EINVAL, 0);
  // 8-bit activations
  EXPECT(gptq_w4a8_matmul(x8, f, 1, 256, q, h, h, 8, 256, 32, 0, f, nullptr, 0, nullptr), GPTQ_OK, 1);
  EXPECT(gptq_w4a8_matmul(x8, f, 200, 256, q, h, h, 8, 256, 32, 0, f, p, 4096, nullptr), GPTQ_OK, 1);
  EXPECT(gptq_w4a8_matmul(x8, f, 200, 256, q, h, h, 8, 256, 32, 0, f, p, 4095, nullptr), GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a8_matmul(x8, f, 200, 256, q, h, h, 8, 256, 32, 0, f, buf + 64, 4096, nullptr),
         GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a8_matmul(x8, f, 200, 256, q, h, h, 8, 256, 32, 0, f, nullptr, 4096, nullptr),
         GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a8_matmul(x8, f, 1, 264, q, h, h, 8, 256, 32, 0, f, nullptr, 0, nullptr), GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a8_matmul(x8, nullptr, 1, 256, q, h, h, 8, 256, 32, 0, f, nullptr, 0, nullptr),
         GPTQ_EINVAL, 0);
  EXPECT(gptq_w4a8_matmul(x8, f, 0, 256, q, h, h, 8, 256, 32, 0, f, nullptr, 0, nullptr), GPTQ_OK, 0);
  EXPECT((int)gptq_w4a8_workspace(200, 8, 256, 32), 4096, 0);
  EXPECT((int)gptq_w4a8_workspace(200, 8, 200, 32), 0, 0);
  EXPECT((int)gptq_w4a8_workspace(-1, 8, 256, 32), 0, 0);
  EXPECT((int)gptq_w4a8_workspace(big, 8, 256, 32), 0, 0);
  // the norm
  EXPECT(gptq_add_rmsnorm(p, 0, 64, p, 0, 64, p, 64, p, 0, 1e-6, 2, 64, p, 2, 64, f, nullptr), GPTQ_OK, 1);
  EXPECT(gptq_add_rmsnorm(p, 1, 64, nullptr, 9, 0, nullptr, 0, p, 1, 0.0, 2, 64, p, 0, 64, nullptr, nullptr),
         GPTQ_OK, 1);
  EXPECT(gptq_add_rmsnorm(p, 1, 64, p, 1, 64, nullptr, 0, p, 1, 0.0, 2, 64, p, 0, 64, nullptr, nullptr),
         GPTQ_OK, 1);
  EXPECT(gptq_add_rmsnorm(p, 0, 64, p, 0, 64, p, 64, p, 0, 1e-6, 0, 64, p, 2, 64, f, nullptr), GPTQ_OK, 0);
  EXPECT(gptq_add_rmsnorm(p, 0, 64, p, 0, 64, p, 64, p, 0, std::nan(""), 2, 64, p, 2, 64, f, nullptr),
         GPTQ_EINVAL, 0);
  EXPECT(gptq_add_rmsnorm(p, 0, 64, nullptr, 0, 64, p, 64, p, 0, 1e-6, 2, 64, p, 2, 64, f, nullptr),
         GPTQ_EINVAL, 0);
  EXPECT(gptq_add_rmsnorm(p, 0, 64, p, 0, 64, p, 72, p, 0, 1e-6, 2, 64, p, 2, 64, f, nullptr),
         GPTQ_EINVAL, 0);
  EXPECT(gptq_add_rmsnorm(p, 0, 64, p, 0, 64, p, 64, p, 0, 1e-6, big, 64, p, 2, 64, f, nullptr),
         GPTQ_EINVAL, 0);
  EXPECT(gptq_add_rmsnorm(p, 0, 64, p, 0, 64, p, 64, p, 0, 1e-6, 2, big, p, 2, 64, f, nullptr),
         GPTQ_EINVAL, 0);
  EXPECT(gptq_add_rmsnorm(p, 0, 64, p, 0, 64, p, 64, p, 0, 1e-6, 2, 64, p, 1, 64, f, nullptr),
         GPTQ_EUNSUPPORTED, 0);
  std::printf("%d checks, %d failed\n", g_checks, g_fails);
  return g_fails != 0;
}
