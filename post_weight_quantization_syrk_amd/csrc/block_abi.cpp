// C ABI front end of the calls that complete a quantized decoder block: the
// 4-bit product with its epilogue, the norms of queries and keys with the
// rotation, and attention.  Every entry point validates its arguments before
// enqueueing anything.
#include <hip/hip_runtime.h>

#include "../../include/gptq.h"
#include "kernels.h"

namespace {

int hip_status(hipError_t e) { return e == hipSuccess ? GPTQ_OK : GPTQ_EHIP; }

bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }

bool workspace(const void* ws, size_t have, size_t need) {
  return have >= need && (need == 0 || (ws && aligned(ws, 256)));
}

bool float_type(int t) { return t == GPTQ_BF16 || t == GPTQ_F32; }

size_t type_size(int t) { return t == GPTQ_F32 ? 4 : 2; }

constexpr int64_t MOST = 1 << 30;
constexpr int64_t MOST_ROWS = (int64_t)1 << 38;  // of a cache: places fit 64 bits

int check_linear(int64_t m, int64_t d_out, int64_t d_in, int group_size, int gated) {
  if (m < 0 || m > MOST || d_out <= 0 || d_out > MOST || d_in <= 0 || d_in > 65536)
    return GPTQ_EINVAL;
  if ((gated != 0 && gated != 1) || (gated && d_out % 2 != 0)) return GPTQ_EINVAL;
  if (group_size != -1 && (group_size <= 0 || d_in % group_size != 0)) return GPTQ_EINVAL;
  if (group_size != -1 && group_size != 32 && group_size != 64 && group_size != 128)
    return GPTQ_EUNSUPPORTED;
  if (d_in % 32 != 0) return GPTQ_EUNSUPPORTED;
  return GPTQ_OK;
}

// Strides between rows and between heads: whole 16-byte pieces, and offsets
// inside a tile of rows that fit 32 bits.
int check_heads(int64_t ld, int64_t hs, size_t size) {
  if (ld < 0 || hs < 0 || ld % (int64_t)(16 / size) != 0 || hs % (int64_t)(16 / size) != 0)
    return GPTQ_EINVAL;
  if (ld >= 1 << 23 || hs >= ((int64_t)1 << 40)) return GPTQ_EUNSUPPORTED;
  return GPTQ_OK;
}

// An output's besides: no two of its values in one place (rows outside heads, or
// heads outside rows).
int check_out(int64_t ld, int64_t hs, int64_t rows, int64_t heads, int64_t hd) {
  const int st = check_heads(ld, hs, 2);
  if (st != GPTQ_OK) return st;
  const bool by_rows = (heads == 1 || hs >= hd) && (rows <= 1 || ld >= (heads - 1) * hs + hd);
  const bool by_heads = (rows <= 1 || ld >= hd) && (heads == 1 || hs >= (rows - 1) * ld + hd);
  return by_rows || by_heads ? GPTQ_OK : GPTQ_EINVAL;
}

int check_attention(int64_t tq, int64_t batch, int64_t hq, int64_t hk, int64_t hd) {
  if (tq < 0 || tq > MOST || batch < 0 || batch > MOST || hq <= 0 || hk <= 0 || hd <= 0)
    return GPTQ_EINVAL;
  if (hq % hk != 0) return GPTQ_EINVAL;
  if (hq > 65536 || hd % 8 != 0 || hd > 256) return GPTQ_EUNSUPPORTED;
  // threads of one launch are below 2^32
  if ((tq * (hq / hk) / 32 + batch) * hk > 1 << 23) return GPTQ_EUNSUPPORTED;
  return GPTQ_OK;
}

}  // namespace

extern "C" {

size_t gptq_w4a16_linear_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size,
                                   int gated) {
  if (m <= 0 || check_linear(m, d_out, d_in, group_size, gated) != GPTQ_OK) return 0;
  return gptq::linear_workspace(m, d_out, d_in, group_size, gated != 0);
}

int gptq_w4a16_linear(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                      const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                      int64_t d_in, int group_size, int sym, const void* bias, int bias_dtype,
                      int activation, int gated, const void* residual, int res_dtype, int64_t ldr,
                      void* Y, int y_dtype, int64_t ldy, void* ws, size_t ws_bytes,
                      gptq_stream stream) {
  const int st = check_linear(m, d_out, d_in, group_size, gated);
  if (st != GPTQ_OK) return st;
  if (sym != 0 && sym != 1) return GPTQ_EINVAL;
  if (activation < GPTQ_ACT_NONE || activation > GPTQ_ACT_GELU_TANH) return GPTQ_EINVAL;
  if (!float_type(y_dtype) || (bias && !float_type(bias_dtype)) ||
      (residual && !float_type(res_dtype)))
    return GPTQ_EINVAL;
  if (m == 0) return GPTQ_OK;
  const int64_t F = gated ? d_out / 2 : d_out;
  if (ldx < d_in || ldx % 8 != 0 || !X || !aligned(X, 16)) return GPTQ_EINVAL;
  if (ldx > 1 << 23) return GPTQ_EUNSUPPORTED;
  if (!qweight || !scales_f16 || (!sym && !zeros_f16) || !aligned(qweight, 16) ||
      !aligned(scales_f16, 2) || !aligned(zeros_f16, 2))
    return GPTQ_EINVAL;
  if (!Y || ldy < F || !aligned(Y, type_size(y_dtype))) return GPTQ_EINVAL;
  if (bias && !aligned(bias, type_size(bias_dtype))) return GPTQ_EINVAL;
  if (residual && (ldr < F || !aligned(residual, type_size(res_dtype)))) return GPTQ_EINVAL;
  if (residual == Y && (ldr != ldy || res_dtype != y_dtype)) return GPTQ_EINVAL;
  if (!workspace(ws, ws_bytes, gptq::linear_workspace(m, d_out, d_in, group_size, gated != 0)))
    return GPTQ_EINVAL;
  gptq::Epilogue e;
  e.bias = bias, e.res = residual, e.y = Y, e.ldr = ldr, e.ldy = ldy, e.F = (int)F;
  e.act = activation;
  e.bias_f32 = bias_dtype == GPTQ_F32, e.res_f32 = res_dtype == GPTQ_F32;
  e.y_f32 = y_dtype == GPTQ_F32;
  e.vec4 = ldy % 4 == 0 && aligned(Y, 4 * type_size(y_dtype));
  return hip_status(gptq::linear_launch(X, m, ldx, qweight, scales_f16, sym ? nullptr : zeros_f16,
                                        d_out, d_in, group_size, gated != 0, e, ws,
                                        (hipStream_t)stream));
}

int gptq_qk_norm_rope(const void* Q, int64_t ldq, int64_t hsq, const void* K, int64_t ldk,
                      int64_t hsk, const void* V, int64_t ldv, int64_t hsv, int x_dtype, int64_t m,
                      int hq, int hk, int hd, const int32_t* positions, const double* inv_freq,
                      int rot_dim, int interleaved, const void* q_weight, const void* k_weight,
                      int w_dtype, double eps, const int64_t* slots, int64_t kv_rows, void* Q_out,
                      int64_t ldqo, int64_t hsqo, void* K_out, int64_t ldko, int64_t hsko,
                      void* V_out, int64_t ldvo, int64_t hsvo, gptq_stream stream) {
  if (m < 0 || m > MOST || hq <= 0 || hk <= 0 || hd <= 0 || rot_dim < 0 || rot_dim > hd ||
      rot_dim % 2 != 0 || kv_rows < 0 || kv_rows > MOST_ROWS)
    return GPTQ_EINVAL;
  if (!float_type(x_dtype) || (interleaved != 0 && interleaved != 1)) return GPTQ_EINVAL;
  if ((q_weight || k_weight) && (!float_type(w_dtype) || !(eps >= 0.0) || !(eps < 1e30)))
    return GPTQ_EINVAL;
  if (hd % 8 != 0 || hd > 256 || rot_dim % 16 != 0 || hq > 65536 || hk > 65536)
    return GPTQ_EUNSUPPORTED;
  // threads of one launch are below 2^32
  if (m * (16 * ((int64_t)hq + 2 * hk) + 64) >> 32) return GPTQ_EUNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  if (!V != !V_out) return GPTQ_EINVAL;
  if (!Q || !K || !Q_out || !K_out) return GPTQ_EINVAL;
  if (rot_dim && (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 8)))
    return GPTQ_EINVAL;
  if (!slots && kv_rows < m) return GPTQ_EINVAL;
  if (slots && !aligned(slots, 8)) return GPTQ_EINVAL;
  const size_t xs = type_size(x_dtype), wsz = type_size(w_dtype);
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(Q_out, 16) ||
      !aligned(K_out, 16) || !aligned(V_out, 16) || !aligned(q_weight, wsz) ||
      !aligned(k_weight, wsz))
    return GPTQ_EINVAL;
  const int64_t kv_used = slots ? kv_rows : m;
  int st = check_heads(ldq, hsq, xs);
  if (st == GPTQ_OK) st = check_heads(ldk, hsk, xs);
  if (st == GPTQ_OK && V) st = check_heads(ldv, hsv, xs);
  if (st == GPTQ_OK) st = check_out(ldqo, hsqo, m, hq, hd);
  if (st == GPTQ_OK) st = check_out(ldko, hsko, kv_used, hk, hd);
  if (st == GPTQ_OK && V) st = check_out(ldvo, hsvo, kv_used, hk, hd);
  if (st != GPTQ_OK) return st;
  gptq::RopeArgs a;
  a.q = Q, a.k = K, a.v = V;
  a.ldq = ldq, a.hsq = hsq, a.ldk = ldk, a.hsk = hsk, a.ldv = ldv, a.hsv = hsv;
  a.m = m, a.hq = hq, a.hk = hk, a.hd = hd, a.rot = rot_dim;
  a.positions = positions, a.inv_freq = inv_freq;
  a.q_weight = q_weight, a.k_weight = k_weight;
  a.w_f32 = w_dtype == GPTQ_F32, a.interleaved = interleaved != 0, a.eps = eps;
  a.slots = slots, a.kv_rows = kv_rows;
  a.q_out = (uint16_t*)Q_out, a.k_out = (uint16_t*)K_out, a.v_out = (uint16_t*)V_out;
  a.ldqo = ldqo, a.hsqo = hsqo, a.ldko = ldko, a.hsko = hsko, a.ldvo = ldvo, a.hsvo = hsvo;
  return hip_status(gptq::qk_norm_rope_launch(a, x_dtype == GPTQ_F32, (hipStream_t)stream));
}

size_t gptq_attention_workspace(int64_t total_q, int64_t batch, int hq, int hk, int hd,
                                int64_t max_kv_len) {
  if (total_q <= 0 || batch <= 0 || max_kv_len < 0 ||
      check_attention(total_q, batch, hq, hk, hd) != GPTQ_OK)
    return 0;
  return gptq::attention_workspace(total_q, batch, hq, hk, hd, max_kv_len);
}

int gptq_attention(const void* Q, int64_t ldq, int64_t hsq, const void* K, int64_t ldk, int64_t hsk,
                   const void* V, int64_t ldv, int64_t hsv, int64_t total_q, int64_t kv_rows,
                   int64_t batch, int hq, int hk, int hd, const int32_t* cu_q,
                   const int64_t* kv_start, const int32_t* kv_len, int64_t max_kv_len, int causal,
                   double scale, void* out, int64_t ldo, int64_t hso, void* ws, size_t ws_bytes,
                   gptq_stream stream) {
  int st = check_attention(total_q, batch, hq, hk, hd);
  if (st != GPTQ_OK) return st;
  if (kv_rows < 0 || kv_rows > MOST_ROWS || max_kv_len < 0 || (causal != 0 && causal != 1)) return GPTQ_EINVAL;
  // (a scale that is 0 in float32 would turn the masked scores' infinities into NaN)
  if (!(scale >= 1e-30) || !(scale < 1e30)) return GPTQ_EINVAL;
  if (!kv_start != !kv_len) return GPTQ_EINVAL;
  if (total_q == 0 || batch == 0) return GPTQ_OK;
  if (!Q || !out || !cu_q || (kv_rows > 0 && (!K || !V))) return GPTQ_EINVAL;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(out, 16) ||
      !aligned(cu_q, 4) || !aligned(kv_start, 8) || !aligned(kv_len, 4))
    return GPTQ_EINVAL;
  st = check_heads(ldq, hsq, 2);
  if (st == GPTQ_OK) st = check_heads(ldk, hsk, 2);
  if (st == GPTQ_OK) st = check_heads(ldv, hsv, 2);
  if (st == GPTQ_OK) st = check_out(ldo, hso, total_q, hq, hd);
  if (st != GPTQ_OK) return st;
  if (!workspace(ws, ws_bytes, gptq::attention_workspace(total_q, batch, hq, hk, hd, max_kv_len)))
    return GPTQ_EINVAL;
  gptq::AttnArgs a;
  a.q = (const uint16_t*)Q, a.k = (const uint16_t*)K, a.v = (const uint16_t*)V;
  a.ldq = ldq, a.hsq = hsq, a.ldk = ldk, a.hsk = hsk, a.ldv = ldv, a.hsv = hsv;
  a.tq = total_q, a.kv_rows = kv_rows, a.batch = (int)batch, a.hq = hq, a.hk = hk, a.hd = hd;
  a.cu_q = cu_q, a.kv_start = kv_start, a.kv_len = kv_len;
  a.causal = causal, a.scale = (float)scale;
  a.out = (uint16_t*)out, a.ldo = ldo, a.hso = hso;
  return hip_status(gptq::attention_launch(a, max_kv_len, ws, (hipStream_t)stream));
}

}  // extern "C"
