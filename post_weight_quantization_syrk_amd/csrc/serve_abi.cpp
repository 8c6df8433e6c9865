// C ABI front end of the calls that run a quantized layer on a few tokens or
// in 8 bits: argument checks, workspace sizing and the launch.  Every entry
// point validates its arguments before enqueueing anything.
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

size_t type_size(int t) { return t == GPTQ_F32 ? 4 : t == GPTQ_BF16 ? 2 : 1; }

// The checks that the two products with packed 4-bit weights share; GPTQ_OK
// when the sizes and the format are supported.
int check_w4(int64_t m, int64_t d_out, int64_t d_in, int group_size, int sym) {
  if (m < 0 || m > (1 << 30) || d_out <= 0 || d_out > (1 << 30) || d_in <= 0 || d_in > 65536)
    return GPTQ_EINVAL;
  if (sym != 0 && sym != 1) return GPTQ_EINVAL;
  if (group_size != -1 && (group_size <= 0 || d_in % group_size != 0)) return GPTQ_EINVAL;
  if (group_size != -1 && group_size != 32 && group_size != 64 && group_size != 128)
    return GPTQ_EUNSUPPORTED;
  if (d_in % 32 != 0) return GPTQ_EUNSUPPORTED;
  return GPTQ_OK;
}

bool w4_pointers(const uint32_t* qweight, const uint16_t* scales_f16, const uint16_t* zeros_f16,
                 int sym, const float* Y) {
  return qweight && scales_f16 && Y && (sym || zeros_f16) && aligned(qweight, 16) &&
         aligned(scales_f16, 2) && aligned(zeros_f16, 2) && aligned(Y, 4);
}

}  // namespace

extern "C" {

int gptq_add_rmsnorm(const void* X, int x_dtype, int64_t ldx, const void* R, int r_dtype,
                     int64_t ldr, void* R_out, int64_t ldro, const void* weight, int w_dtype,
                     double eps, int64_t m, int64_t d, void* out, int out_dtype, int64_t ldo,
                     float* out_scales, gptq_stream stream) {
  if (m < 0 || m > (1 << 30) || d <= 0 || d > 65536) return GPTQ_EINVAL;
  if (!float_type(x_dtype) || !float_type(w_dtype)) return GPTQ_EINVAL;
  if (R && !float_type(r_dtype)) return GPTQ_EINVAL;
  if (out_dtype != GPTQ_BF16 && out_dtype != GPTQ_I8)
    return out_dtype == GPTQ_F32 ? GPTQ_EUNSUPPORTED : GPTQ_EINVAL;
  if (!(eps >= 0.0) || !(eps < 1e30)) return GPTQ_EINVAL;
  if (R_out && !R) return GPTQ_EINVAL;
  if (m == 0) return GPTQ_OK;
  if (ldx < d || ldo < d || (R && ldr < d) || (R_out && ldro < d)) return GPTQ_EINVAL;
  if (!X || !weight || !out || (out_dtype == GPTQ_I8 && !out_scales)) return GPTQ_EINVAL;
  if (!aligned(X, type_size(x_dtype)) || !aligned(weight, type_size(w_dtype)) ||
      !aligned(out, type_size(out_dtype)) || !aligned(out_scales, 4))
    return GPTQ_EINVAL;
  if (R && (!aligned(R, type_size(r_dtype)) || !aligned(R_out, type_size(r_dtype))))
    return GPTQ_EINVAL;
  if (R_out == R && R && ldro != ldr) return GPTQ_EINVAL;
  return hip_status(gptq::add_rmsnorm_launch(X, x_dtype, ldx, R, r_dtype, ldr, R_out, ldro, weight,
                                             w_dtype, eps, m, d, out, out_dtype, ldo, out_scales,
                                             (hipStream_t)stream));
}

size_t gptq_w4a16_matvec_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size) {
  if (m <= 0 || m > GPTQ_MATVEC_MAX_M || check_w4(m, d_out, d_in, group_size, 0) != GPTQ_OK)
    return 0;
  return gptq::w4a16_vec_workspace(m, d_out, d_in, group_size);
}

int gptq_w4a16_matvec(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                      const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                      int64_t d_in, int group_size, int sym, float* Y, void* ws, size_t ws_bytes,
                      gptq_stream stream) {
  const int st = check_w4(m, d_out, d_in, group_size, sym);
  if (st != GPTQ_OK) return st;
  if (m > GPTQ_MATVEC_MAX_M) return GPTQ_EUNSUPPORTED;
  if (m == 0) return GPTQ_OK;
  if (ldx < d_in || ldx % 8 != 0 || !X || !aligned(X, 16)) return GPTQ_EINVAL;
  if (!w4_pointers(qweight, scales_f16, zeros_f16, sym, Y)) return GPTQ_EINVAL;
  if (!workspace(ws, ws_bytes, gptq::w4a16_vec_workspace(m, d_out, d_in, group_size)))
    return GPTQ_EINVAL;
  return hip_status(gptq::w4a16_vec_launch(X, m, ldx, qweight, scales_f16,
                                           sym ? nullptr : zeros_f16, d_out, d_in, group_size, Y,
                                           ws, (hipStream_t)stream));
}

size_t gptq_w4a8_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size) {
  if (m <= 0 || check_w4(m, d_out, d_in, group_size, 0) != GPTQ_OK) return 0;
  return gptq::w4a8_workspace(m, d_out, d_in, group_size);
}

int gptq_w4a8_matmul(const int8_t* X, const float* x_scales, int64_t m, int64_t ldx,
                     const uint32_t* qweight, const uint16_t* scales_f16,
                     const uint16_t* zeros_f16, int64_t d_out, int64_t d_in, int group_size,
                     int sym, float* Y, void* ws, size_t ws_bytes, gptq_stream stream) {
  const int st = check_w4(m, d_out, d_in, group_size, sym);
  if (st != GPTQ_OK) return st;
  if (m == 0) return GPTQ_OK;
  if (ldx < d_in || ldx % 16 != 0 || !X || !aligned(X, 16)) return GPTQ_EINVAL;
  if (!x_scales || !aligned(x_scales, 4)) return GPTQ_EINVAL;
  if (!w4_pointers(qweight, scales_f16, zeros_f16, sym, Y)) return GPTQ_EINVAL;
  if (!workspace(ws, ws_bytes, gptq::w4a8_workspace(m, d_out, d_in, group_size)))
    return GPTQ_EINVAL;
  return hip_status(gptq::w4a8_launch(X, x_scales, m, ldx, qweight, scales_f16,
                                      sym ? nullptr : zeros_f16, d_out, d_in, group_size, Y, ws,
                                      (hipStream_t)stream));
}

}  // extern "C"
