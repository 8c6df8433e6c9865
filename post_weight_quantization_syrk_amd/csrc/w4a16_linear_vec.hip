// The W4A16 product with its epilogue for a few tokens (m <= 64).
#include "kernels.h"
#include "w4_dot.h"

namespace gptq {

size_t linear_vec_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size, bool gated) {
  const int G = group_size == -1 ? 0 : group_size;
  return w4vec::dot_takes(m, d_in) ? 0 : w4vec::vec_plan(false, m, d_out, d_in, G, true, gated).ws_bytes;
}

hipError_t linear_vec_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                             const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                             int64_t d_in, int group_size, bool gated, const Epilogue& e, void* ws,
                             hipStream_t stream) {
  w4vec::VecArgs a;
  a.x = (const char*)X, a.sx = nullptr, a.q = qweight, a.s16 = scales_f16, a.z16 = zeros_f16;
  a.y = nullptr, a.ldx = 2 * ldx, a.m = (int)m, a.n = (int)d_out, a.k = (int)d_in;
  a.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
  a.vec = w4vec::scale_vec(scales_f16, zeros_f16, a.ng);
  a.splits = 1, a.per_split = 0, a.slots = 0;
  const int G = group_size == -1 ? 0 : group_size;
  if (w4vec::dot_takes(m, d_in))
    return gated ? w4vec::dot_launch<false>(a, G, stream, w4vec::Finished<true>{e})
                 : w4vec::dot_launch<false>(a, G, stream, w4vec::Finished<false>{e});
  return gated ? w4vec::vec_finish_launch<false, true>(a, G, ws, e, stream)
               : w4vec::vec_finish_launch<false, false>(a, G, ws, e, stream);
}

}  // namespace gptq
