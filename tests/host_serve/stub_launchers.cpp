// Host-only stand-ins for the launchers behind serve_abi.cpp: each checks what
// the front end promises before it launches, and counts the calls.
#include <cstdio>
#include <cstdlib>

#include "kernels.h"

int g_launches = 0;

namespace {
void need(bool ok, const char* what) {
  if (!ok) {
    std::fprintf(stderr, "stub launcher: front end broke its promise: %s\n", what);
    std::abort();
  }
}
bool to(const void* p, size_t n) { return p && (uintptr_t)p % n == 0; }
}  // namespace

namespace gptq {

size_t w4a16_vec_workspace(int64_t m, int64_t d_out, int64_t d_in, int) {
  need(m > 0 && m <= 64 && d_out > 0 && d_in > 0, "w4a16_vec_workspace sizes");
  return m > 32 ? 2048 : 0;
}
hipError_t w4a16_vec_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                            const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                            int64_t d_in, int group_size, float* Y, void* ws, hipStream_t) {
  need(to(X, 16) && to(qweight, 16) && to(scales_f16, 2) && to(Y, 4), "w4a16_vec pointers");
  need(m <= 32 || to(ws, 256), "workspace");
  need(m > 0 && m <= 64 && d_out > 0 && d_in > 0 && d_in % 32 == 0 && d_in <= 65536, "sizes");
  need(ldx >= d_in && ldx % 8 == 0, "ldx");
  need(group_size == -1 || d_in % group_size == 0, "group");
  (void)zeros_f16;
  ++g_launches;
  return hipSuccess;
}
size_t w4a8_workspace(int64_t m, int64_t d_out, int64_t d_in, int) {
  need(m > 0 && d_out > 0 && d_in > 0, "w4a8_workspace sizes");
  return m > 100 ? 4096 : 0;
}
hipError_t w4a8_launch(const int8_t* X, const float* x_scales, int64_t m, int64_t ldx,
                       const uint32_t* qweight, const uint16_t* scales_f16, const uint16_t*,
                       int64_t d_out, int64_t d_in, int group_size, float* Y, void* ws,
                       hipStream_t) {
  need(to(X, 16) && to(x_scales, 4) && to(qweight, 16) && to(scales_f16, 2) && to(Y, 4), "w4a8");
  need(m > 0 && d_out > 0 && d_in > 0 && d_in % 32 == 0 && d_in <= 65536, "sizes");
  need(ldx >= d_in && ldx % 16 == 0, "ldx");
  need(group_size == -1 || d_in % group_size == 0, "group");
  need(m <= 100 || to(ws, 256), "workspace");
  ++g_launches;
  return hipSuccess;
}
hipError_t add_rmsnorm_launch(const void* X, int x_dtype, int64_t ldx, const void* R, int r_dtype,
                              int64_t ldr, void* R_out, int64_t ldro, const void* weight,
                              int w_dtype, double eps, int64_t m, int64_t d, void* out,
                              int out_dtype, int64_t ldo, float* out_scales, hipStream_t) {
  need(X && weight && out && m > 0 && d > 0 && d <= 65536 && eps >= 0.0, "add_rmsnorm");
  need(x_dtype <= 1 && w_dtype <= 1 && (!R || r_dtype <= 1), "types");
  need(ldx >= d && ldo >= d && (!R || ldr >= d) && (!R_out || (R && ldro >= d)), "strides");
  need(out_dtype == 0 || (out_dtype == 2 && out_scales), "output");
  ++g_launches;
  return hipSuccess;
}

}  // namespace gptq
