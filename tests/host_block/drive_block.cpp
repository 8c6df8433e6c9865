// Drives the entry points of block_abi.cpp through accepted and rejected
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
#define EXPECT(call, want, launches)                                      \
  do {                                                                    \
    const int before = g_launches;                                        \
    const int got = (call);                                               \
    check(got, (want), g_launches - before, (launches), #call, __LINE__); \
  } while (0)
}  // namespace

int main() {
  alignas(256) static unsigned char buf[4096];
  void* p = buf;
  auto* q = (uint32_t*)p;
  auto* h = (uint16_t*)p;
  auto* i32 = (int32_t*)p;
  auto* i64 = (int64_t*)p;
  auto* d = (double*)p;
  const int64_t big = std::numeric_limits<int64_t>::max();
  const double nan = std::nan("");
  auto linear = [&](int64_t m, int64_t d_out, int64_t d_in, int g, int gated, const void* bias, int act,
                    const void* res, int rt, int64_t ldr, void* y, int yt, int64_t ldy, size_t ws) {
    return gptq_w4a16_linear(p, m, 256, q, h, h, d_out, d_in, g, 0, bias, 0, act, gated, res, rt, ldr, y,
                             yt, ldy, ws ? p : nullptr, ws, nullptr);
  };
  EXPECT(linear(1, 8, 256, 128, 0, nullptr, 0, nullptr, 0, 0, p, 0, 8, 0), GPTQ_OK, 1);
  EXPECT(linear(64, 8, 256, -1, 1, p, 4, p, 1, 4, p, 1, 4, 0), GPTQ_OK, 1);
  EXPECT(linear(65, 8, 256, 32, 0, p, 1, p, 0, 9, buf + 2, 0, 9, 4096), GPTQ_OK, 1);
  EXPECT(linear(65, 8, 256, 32, 0, p, 1, p, 0, 9, p, 0, 9, 4095), GPTQ_EINVAL, 0);
  EXPECT(linear(65, 8, 256, 32, 0, p, 1, p, 0, 8, p, 0, 9, 4096), GPTQ_EINVAL, 0);
  EXPECT(linear(65, 7, 256, 32, 1, p, 1, p, 0, 8, p, 0, 8, 4096), GPTQ_EINVAL, 0);
  EXPECT(linear(0, 8, 256, 32, 0, p, 1, p, 0, 8, p, 0, 8, 0), GPTQ_OK, 0);
  EXPECT(linear(big, 8, 256, 32, 0, p, 1, p, 0, 8, p, 0, 8, 0), GPTQ_EINVAL, 0);
  EXPECT(linear(1, big, 256, 32, 0, p, 1, p, 0, 8, p, 0, 8, 0), GPTQ_EINVAL, 0);
  EXPECT(linear(1, 8, big, 32, 0, p, 1, p, 0, 8, p, 0, 8, 0), GPTQ_EINVAL, 0);
  EXPECT(linear(1, 8, 256, 256, 0, p, 1, p, 0, 8, p, 0, 8, 0), GPTQ_EUNSUPPORTED, 0);
  EXPECT(linear(1, 8, 256, 32, 0, p, 9, p, 0, 8, p, 0, 8, 0), GPTQ_EINVAL, 0);
  EXPECT((int)gptq_w4a16_linear_workspace(65, 8, 256, 32, 0), 4096, 0);
  EXPECT((int)gptq_w4a16_linear_workspace(-1, 8, 256, 32, 0), 0, 0);
  EXPECT((int)gptq_w4a16_linear_workspace(65, 7, 256, 32, 1), 0, 0);
  EXPECT((int)gptq_w4a16_linear_workspace(big, big, big, 32, 1), 0, 0);

  auto rope = [&](int64_t m, int hq, int hk, int hd, int rot, const int64_t* slots, int64_t rows, double eps,
                  void* v, int64_t ldq, int64_t ldqo) {
    return gptq_qk_norm_rope(p, ldq, hd, p, hk * hd, hd, v, hk * hd, hd, 0, m, hq, hk, hd, i32, d, rot, 0, p,
                             nullptr, 0, eps, slots, rows, p, ldqo, hd, p, hk * hd, hd, v, hk * hd, hd, nullptr);
  };
  EXPECT(rope(4, 8, 2, 64, 64, nullptr, 4, 0.0, nullptr, 512, 512), GPTQ_OK, 1);
  EXPECT(rope(4, 8, 2, 64, 0, i64, 0, 1e-5, p, 0, 512), GPTQ_OK, 1);
  EXPECT(rope(4, 8, 2, 64, 64, nullptr, 3, 0.0, p, 512, 512), GPTQ_EINVAL, 0);
  EXPECT(rope(4, 8, 2, 64, 64, nullptr, 4, nan, p, 512, 512), GPTQ_EINVAL, 0);
  EXPECT(rope(4, 8, 2, 64, 64, nullptr, 4, 0.0, p, 512, 504), GPTQ_EINVAL, 0);
  EXPECT(rope(4, 8, 2, 64, 64, nullptr, 4, 0.0, p, big, 512), GPTQ_EINVAL, 0);
  EXPECT(rope(4, 8, 2, 64, 24, nullptr, 4, 0.0, p, 512, 512), GPTQ_EUNSUPPORTED, 0);
  EXPECT(rope(4, 8, 2, 65, 64, nullptr, 4, 0.0, p, 512, 512), GPTQ_EUNSUPPORTED, 0);
  EXPECT(rope(0, 8, 2, 64, 64, nullptr, 4, 0.0, p, 512, 512), GPTQ_OK, 0);
  EXPECT(rope(big, 8, 2, 64, 64, i64, 4, 0.0, p, 512, 512), GPTQ_EINVAL, 0);

  auto attention = [&](int64_t tq, int64_t rows, int64_t batch, int hq, int hk, int hd, const int64_t* start,
                       const int32_t* len, int64_t longest, double scale, int64_t ldo, size_t ws) {
    return gptq_attention(p, hq * hd, hd, p, hk * hd, hd, p, hk * hd, hd, tq, rows, batch, hq, hk, hd, i32,
                          start, len, longest, 1, scale, p, ldo, hd, ws ? p : nullptr, ws, nullptr);
  };
  EXPECT(attention(10, 10, 2, 8, 2, 64, nullptr, nullptr, 10, 0.1, 512, 0), GPTQ_OK, 1);
  EXPECT(attention(10, 5000, 2, 8, 2, 64, i64, i32, 5000, 0.1, 512, 8192), GPTQ_OK, 1);
  EXPECT(attention(10, 5000, 2, 8, 2, 64, i64, i32, 5000, 0.1, 512, 8191), GPTQ_EINVAL, 0);
  EXPECT(attention(10, 10, 2, 8, 2, 64, i64, nullptr, 10, 0.1, 512, 0), GPTQ_EINVAL, 0);
  EXPECT(attention(10, 10, 2, 8, 3, 64, i64, i32, 10, 0.1, 512, 0), GPTQ_EINVAL, 0);
  EXPECT(attention(10, 10, 2, 8, 2, 64, i64, i32, 10, nan, 512, 0), GPTQ_EINVAL, 0);
  EXPECT(attention(10, 10, 2, 8, 2, 64, i64, i32, 10, 0.1, 504, 0), GPTQ_EINVAL, 0);
  EXPECT(attention(10, 10, 2, 8, 2, 66, i64, i32, 10, 0.1, 528, 0), GPTQ_EUNSUPPORTED, 0);
  EXPECT(attention(1 << 30, 10, 2, 8, 2, 64, i64, i32, 10, 0.1, 512, 0), GPTQ_EUNSUPPORTED, 0);
  EXPECT(attention(big, 10, 2, 8, 2, 64, i64, i32, 10, 0.1, 512, 0), GPTQ_EINVAL, 0);
  EXPECT(attention(10, 10, big, 8, 2, 64, i64, i32, 10, 0.1, 512, 0), GPTQ_EINVAL, 0);
  EXPECT(attention(0, 10, 2, 8, 2, 64, i64, i32, 10, 0.1, 512, 0), GPTQ_OK, 0);
  EXPECT(attention(10, 10, 0, 8, 2, 64, i64, i32, 10, 0.1, 512, 0), GPTQ_OK, 0);
  EXPECT((int)gptq_attention_workspace(10, 2, 8, 2, 64, 5000), 8192, 0);
  EXPECT((int)gptq_attention_workspace(10, 2, 8, 3, 64, 5000), 0, 0);
  EXPECT((int)gptq_attention_workspace(big, big, 8, 2, 64, big), 0, 0);
  std::printf("%d checks, %d failed\n", g_checks, g_fails);
  return g_fails != 0;
}
