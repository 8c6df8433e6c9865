// The W4A16 product for a few tokens (m <= 64), X bf16.
#include "kernels.h"
#include "w4_dot.h"

namespace gptq {

size_t w4a16_vec_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size) {
  const int G = group_size == -1 ? 0 : group_size;
  return w4vec::dot_takes(m, d_in) ? 0 : w4vec::vec_plan(false, m, d_out, d_in, G).ws_bytes;
}

hipError_t w4a16_vec_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                            const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                            int64_t d_in, int group_size, float* Y, void* ws,
                            hipStream_t stream) {
  w4vec::VecArgs a;
  a.x = (const char*)X, a.sx = nullptr, a.q = qweight, a.s16 = scales_f16, a.z16 = zeros_f16;
  a.y = Y, a.ldx = 2 * ldx, a.m = (int)m, a.n = (int)d_out, a.k = (int)d_in;
  a.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
  a.vec = w4vec::scale_vec(scales_f16, zeros_f16, a.ng);
  const int G = group_size == -1 ? 0 : group_size;
  return w4vec::dot_takes(m, d_in) ? w4vec::dot_launch<false>(a, G, stream)
                                        : w4vec::vec_launch<false>(a, G, ws, stream);
}

}  // namespace gptq
