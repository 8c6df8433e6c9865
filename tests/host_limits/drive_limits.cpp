// The largest calls that block_abi.cpp accepts, and the smallest past them that it refuses.
// The stand-in launchers check that no launch of an accepted call reaches 2^32 threads.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "gptq.h"
#include "kernels.h"

static int g_launches = 0, g_fails = 0, g_checks = 0;

static void need(bool ok, const char* what) {
  if (!ok) {
    std::fprintf(stderr, "an accepted call would not launch: %s\n", what);
    std::abort();
  }
}

namespace gptq {

size_t linear_workspace(int64_t, int64_t, int64_t, int, bool) { return 0; }
hipError_t linear_launch(const void*, int64_t m, int64_t ldx, const uint32_t*, const uint16_t*, const uint16_t*,
                         int64_t d_out, int64_t d_in, int, bool, const Epilogue& e, void*, hipStream_t) {
  // 32-bit offsets in bytes inside a tile of 256 rows of X
  need(255 * (2 * ldx) + 2 * d_in < (int64_t)1 << 32, "offsets of a tile of X");
  need(m <= 1 << 30 && d_out <= 1 << 30 && e.F <= 1 << 30, "sizes in 32 bits");
  ++g_launches;
  return hipSuccess;
}
hipError_t qk_norm_rope_launch(const RopeArgs& a, bool, hipStream_t) {
  // a wave takes four heads or more, a token at least one wave; four waves to a workgroup
  const int64_t heads = a.hq + a.hk + (a.v ? a.hk : 0), waves = a.m * ((heads + 3) / 4);
  need((waves + 3) / 4 * 256 < (int64_t)1 << 32, "threads");
  ++g_launches;
  return hipSuccess;
}
size_t attention_workspace(int64_t, int64_t, int, int, int, int64_t) { return 0; }
hipError_t attention_launch(const AttnArgs& a, int64_t, void*, hipStream_t) {
  // a tile of 32 rows at the least, and one that is not full for each sequence, of 256 threads
  const int64_t tiles = a.tq * (a.hq / a.hk) / 32 + a.batch;
  need(tiles * a.hk * 256 < (int64_t)1 << 32, "threads");
  need(tiles * a.hk <= 1 << 23, "workgroups");
  need(a.tq * (a.hq / a.hk) < (int64_t)1 << 31, "rows in 32 bits");
  need(64 * 2 * a.ldk < (int64_t)1 << 32 && 64 * 2 * a.ldv < (int64_t)1 << 32, "offsets of a tile of keys");
  ++g_launches;
  return hipSuccess;
}

}  // namespace gptq

static void expect(int got, int want, int launched, const char* what) {
  ++g_checks;
  if (got != want || launched != (want == GPTQ_OK)) {
    std::printf("FAIL: %s returned %d (want %d), launched %d\n", what, got, want, launched);
    ++g_fails;
  }
}
#define EXPECT(call, want)                           \
  do {                                               \
    const int before = g_launches;                   \
    const int got = (call);                          \
    expect(got, (want), g_launches - before, #call); \
  } while (0)

int main() {
  alignas(256) static unsigned char buf[4096];
  void* p = buf;
  auto* q = (uint32_t*)p;
  auto* h = (uint16_t*)p;
  auto* i32 = (int32_t*)p;
  auto* i64 = (int64_t*)p;
  auto* d = (double*)p;
  const int64_t one = 1;

  auto attention = [&](int64_t tq, int64_t batch, int hq, int hk, int64_t ld, int64_t rows) {
    return gptq_attention(p, hq * 64, 64, p, ld, 64, p, ld, 64, tq, rows, batch, hq, hk, 64, i32, i64, i32, 100, 1,
                          0.1, p, hq * 64, 64, nullptr, 0, nullptr);
  };
  // (tq (hq / hk) / 32 + batch) hk up to 2^23
  EXPECT(attention(one << 27, one << 22, 1, 1, 64, 1000), GPTQ_OK);
  EXPECT(attention((one << 27) + 31, one << 22, 1, 1, 64, 1000), GPTQ_OK);
  EXPECT(attention((one << 27) + 32, one << 22, 1, 1, 64, 1000), GPTQ_EUNSUPPORTED);
  EXPECT(attention(one << 27, (one << 22) + 1, 1, 1, 64, 1000), GPTQ_EUNSUPPORTED);
  EXPECT(attention(1, one << 23, 1, 1, 64, 1000), GPTQ_OK);
  EXPECT(attention(1, (one << 23) + 1, 1, 1, 64, 1000), GPTQ_EUNSUPPORTED);
  EXPECT(attention(32, (one << 20) - 8, 64, 8, 512, 1000), GPTQ_OK);
  EXPECT(attention(32, (one << 20) - 7, 64, 8, 512, 1000), GPTQ_EUNSUPPORTED);
  EXPECT(attention(16, 1, 65536, 65536, 64, 1000), GPTQ_OK);
  EXPECT(attention(16, 128, 65536, 65536, 64, 1000), GPTQ_OK);
  EXPECT(attention(16, 129, 65536, 65536, 64, 1000), GPTQ_EUNSUPPORTED);
  EXPECT(attention(16, 1, 65537, 65537, 64, 1000), GPTQ_EUNSUPPORTED);
  EXPECT(attention(1, 1, 1, 1, (one << 23) - 8, 1000), GPTQ_OK);
  EXPECT(attention(1, 1, 1, 1, one << 23, 1000), GPTQ_EUNSUPPORTED);
  EXPECT(attention(1, 1, 1, 1, 64, one << 38), GPTQ_OK);
  EXPECT(attention(1, 1, 1, 1, 64, (one << 38) + 1), GPTQ_EINVAL);

  auto rope = [&](int64_t m, int hq, int hk, int64_t ldq, int64_t rows) {
    return gptq_qk_norm_rope(p, ldq, 64, p, hk * 64, 64, p, hk * 64, 64, 0, m, hq, hk, 64, i32, d, 64, 0, p, p, 0, 1e-6,
                             i64, rows, p, hq * 64, 64, p, hk * 64, 64, p, hk * 64, 64, nullptr);
  };
  // m (16 (hq + 2 hk) + 64) below 2^32
  EXPECT(rope(((one << 32) - 1) / 112, 1, 1, 64, 5), GPTQ_OK);
  EXPECT(rope(((one << 32) - 1) / 112 + 1, 1, 1, 64, 5), GPTQ_EUNSUPPORTED);
  EXPECT(rope(((one << 32) - 1) / 832, 32, 8, 2048, 5), GPTQ_OK);
  EXPECT(rope(((one << 32) - 1) / 832 + 1, 32, 8, 2048, 5), GPTQ_EUNSUPPORTED);
  EXPECT(rope(1300, 65536, 65536, 65536 * 64, 5), GPTQ_OK);
  EXPECT(rope(1, 65537, 1, 65536 * 64, 5), GPTQ_EUNSUPPORTED);
  EXPECT(rope(1, 1, 1, (one << 23) - 8, 5), GPTQ_OK);
  EXPECT(rope(1, 1, 1, one << 23, 5), GPTQ_EUNSUPPORTED);
  EXPECT(rope(1, 1, 1, 64, one << 38), GPTQ_OK);
  EXPECT(rope(1, 1, 1, 64, (one << 38) + 1), GPTQ_EINVAL);

  auto linear = [&](int64_t m, int64_t d_out, int64_t d_in, int64_t ldx) {
    return gptq_w4a16_linear(p, m, ldx, q, h, h, d_out, d_in, 32, 0, nullptr, 0, 0, 0, nullptr, 0, 0, p, 0, d_out,
                             nullptr, 0, nullptr);
  };
  EXPECT(linear(one << 30, 8, 256, 256), GPTQ_OK);
  EXPECT(linear((one << 30) + 1, 8, 256, 256), GPTQ_EINVAL);
  EXPECT(linear(8, one << 30, 256, 256), GPTQ_OK);
  EXPECT(linear(8, (one << 30) + 1, 256, 256), GPTQ_EINVAL);
  EXPECT(linear(8, 8, 65536, 65536), GPTQ_OK);
  EXPECT(linear(8, 8, 65568, 65568), GPTQ_EINVAL);
  EXPECT(linear(300, 8, 65536, one << 23), GPTQ_OK);
  EXPECT(linear(300, 8, 65536, (one << 23) + 8), GPTQ_EUNSUPPORTED);
  std::printf("%d checks, %d failed\n", g_checks, g_fails);
  return g_fails != 0;
}
