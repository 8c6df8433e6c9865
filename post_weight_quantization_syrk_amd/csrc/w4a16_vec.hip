// The W4A16 product for a few tokens (m <= 64):
//   Y[i][n] = sum_k X[i][k] s[n][k/g] (q[n][k] - z[n][k/g])
// A wave per output row; its lanes take the row's packed words in turn, and
// four tokens share a word's codes.
#include "common.h"
#include "kernels.h"

#include <hip/hip_fp16.h>

namespace gptq {

namespace {

constexpr int MT = 4;  // tokens per wave

__global__ __launch_bounds__(256) void w4a16_vec_kernel(const uint16_t* __restrict__ X,
                                                        int64_t ldx, int M, int N, int K,
                                                        const uint32_t* __restrict__ Q,
                                                        const uint16_t* __restrict__ S16,
                                                        const uint16_t* __restrict__ Z16, int G,
                                                        float* __restrict__ Y) {
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int i0 = blockIdx.y * MT;
  if (n >= N) return;
  const int words = K / 8, ng = K / G;
  const uint32_t* q = Q + n * words;
  float tot[MT] = {};
  for (int w = lane; w < words; w += 64) {
    const uint32_t v = q[w];
    const int g = 8 * w / G;
    const float s = __half2float(__ushort_as_half(S16[n * ng + g]));
    const float z = Z16 ? __half2float(__ushort_as_half(Z16[n * ng + g])) : 8.0f;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (i0 + t >= M) break;
      const uint16_t* x = X + (int64_t)(i0 + t) * ldx + 8 * w;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        sum = fmaf(bf16_bits_to_float(x[j]), (float)((v >> (4 * j)) & 15u) - z, sum);
      tot[t] = fmaf(s, sum, tot[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    float v = tot[t];
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if (lane == 0 && i0 + t < M) Y[(int64_t)(i0 + t) * N + n] = v;
  }
}

}  // namespace

hipError_t w4a16_vec_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                            const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                            int64_t d_in, int group_size, float* Y, hipStream_t stream) {
  const int G = group_size == -1 ? (int)d_in : group_size;
  const dim3 grid((unsigned)ceil_div(d_out, 4), (unsigned)ceil_div(m, MT));
  hipLaunchKernelGGL(w4a16_vec_kernel, grid, dim3(256), 0, stream, (const uint16_t*)X, ldx, (int)m,
                     (int)d_out, (int)d_in, qweight, scales_f16, zeros_f16, G, Y);
  return hipGetLastError();
}

}  // namespace gptq
