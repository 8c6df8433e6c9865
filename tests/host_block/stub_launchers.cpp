// Host-only stand-ins for the launchers behind block_abi.cpp: each checks what
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
bool strides(int64_t ld, int64_t hs, int64_t unit) {
  return ld >= 0 && hs >= 0 && ld % unit == 0 && hs % unit == 0 && ld < 1 << 23;
}
}  // namespace

namespace gptq {

size_t linear_workspace(int64_t m, int64_t d_out, int64_t d_in, int, bool gated) {
  need(m > 0 && d_out > 0 && d_in > 0 && (!gated || d_out % 2 == 0), "linear_workspace sizes");
  return m > 64 ? 4096 : 0;
}
hipError_t linear_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                         const uint16_t* scales_f16, const uint16_t*, int64_t d_out, int64_t d_in,
                         int group_size, bool gated, const Epilogue& e, void* ws, hipStream_t) {
  need(to(X, 16) && to(qweight, 16) && to(scales_f16, 2), "linear pointers");
  need(m > 0 && d_out > 0 && d_in > 0 && d_in % 32 == 0 && d_in <= 65536, "sizes");
  need(ldx >= d_in && ldx % 8 == 0, "ldx");
  need(group_size == -1 || d_in % group_size == 0, "group");
  need(e.F == (gated ? d_out / 2 : d_out) && e.ldy >= e.F && to(e.y, e.y_f32 ? 4 : 2), "Y");
  need(!e.res || (e.ldr >= e.F && to(e.res, e.res_f32 ? 4 : 2)), "residual");
  need(!e.bias || to(e.bias, e.bias_f32 ? 4 : 2), "bias");
  need(e.act >= ACT_NONE && e.act <= ACT_GELU_TANH, "activation");
  need(!e.vec4 || (e.ldy % 4 == 0 && to(e.y, e.y_f32 ? 16 : 8)), "vec4");
  need(m <= 64 || to(ws, 256), "workspace");
  ++g_launches;
  return hipSuccess;
}
hipError_t qk_norm_rope_launch(const RopeArgs& a, bool f32, hipStream_t) {
  need(to(a.q, 16) && to(a.k, 16) && to(a.q_out, 16) && to(a.k_out, 16), "rope pointers");
  need(!a.v == !a.v_out, "V and V_out");
  need(a.m > 0 && a.hq > 0 && a.hk > 0 && a.hd > 0 && a.hd % 8 == 0 && a.hd <= 256, "sizes");
  need(a.rot % 16 == 0 && a.rot >= 0 && a.rot <= a.hd && (!a.rot || (a.positions && a.inv_freq)), "rot");
  need(a.slots || a.kv_rows >= a.m, "rows");
  const int unit = f32 ? 4 : 8;
  need(strides(a.ldq, a.hsq, unit) && strides(a.ldk, a.hsk, unit) && strides(a.ldqo, a.hsqo, 8) &&
           strides(a.ldko, a.hsko, 8), "strides");
  need(!a.v || (strides(a.ldv, a.hsv, unit) && strides(a.ldvo, a.hsvo, 8)), "V's strides");
  ++g_launches;
  return hipSuccess;
}
size_t attention_workspace(int64_t tq, int64_t batch, int hq, int hk, int hd, int64_t max_kv_len) {
  need(tq > 0 && batch > 0 && hq > 0 && hk > 0 && hq % hk == 0 && hd > 0 && max_kv_len >= 0,
       "attention_workspace sizes");
  return max_kv_len > 1000 ? 8192 : 0;
}
hipError_t attention_launch(const AttnArgs& a, int64_t max_kv_len, void* ws, hipStream_t) {
  need(to(a.q, 16) && to(a.out, 16) && to(a.cu_q, 4), "attention pointers");
  need(a.kv_rows == 0 || (to(a.k, 16) && to(a.v, 16)), "keys and values");
  need(!a.kv_start == !a.kv_len, "runs of keys");
  need(a.tq > 0 && a.batch > 0 && a.hq % a.hk == 0 && a.hd % 8 == 0 && a.hd <= 256, "sizes");
  need((a.tq * (a.hq / a.hk) / 32 + a.batch) * a.hk <= (int64_t)1 << 25, "grid");
  need(strides(a.ldq, a.hsq, 8) && strides(a.ldk, a.hsk, 8) && strides(a.ldv, a.hsv, 8) &&
           strides(a.ldo, a.hso, 8), "strides");
  need(a.scale > 0.0f, "scale");
  need(max_kv_len <= 1000 || to(ws, 256), "workspace");
  ++g_launches;
  return hipSuccess;
}

}  // namespace gptq
