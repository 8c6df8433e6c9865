// Residual addition, root-mean-square norm, and an output in bf16 or in 8 bits
// with a scale per row:
//   h = x + r (fp32, rounded to r's type),  y_c = h_c w_c / sqrt(mean h^2 + eps)
//   8 bits: p_c = h_c w_c, P = max |p_c|, q_c = rint(127 p_c / P),
//           scale = P / sqrt(mean h^2 + eps) / 127
// The norm's own factor cancels in the codes, so they depend on no sum's
// order; p is exact in float64 and the quotient is formed there.
#include "common.h"
#include "kernels.h"

#include "../../include/gptq.h"

namespace gptq {

namespace {

struct NormArgs {
  const void* X;
  const void* R;
  void* R_out;
  const void* weight;
  void* out;
  float* out_scales;
  int64_t ldx, ldr, ldro, ldo;
  double eps;
  int d;
  int x_f32, r_f32, w_f32, out_i8;
};

__device__ __forceinline__ uint16_t float_to_bf16_bits(float f) {
  const __bf16 b = (__bf16)f;  // nearest, ties to even
  uint16_t u;
  __builtin_memcpy(&u, &b, 2);
  return u;
}

__device__ __forceinline__ float load_as_float(const void* p, int64_t i, int f32) {
  return f32 ? ((const float*)p)[i] : bf16_bits_to_float(((const uint16_t*)p)[i]);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}

// One workgroup of 256 threads per row; h is formed twice.
__global__ __launch_bounds__(256) void add_rmsnorm_kernel(NormArgs a) {
  __shared__ double red[2][4];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  auto h_at = [&](int c) {
    float h = load_as_float(a.X, row * a.ldx + c, a.x_f32);
    if (a.R) {
      h += load_as_float(a.R, row * a.ldr + c, a.r_f32);
      if (!a.r_f32) h = bf16_bits_to_float(float_to_bf16_bits(h));
    }
    return h;
  };
  double sum = 0.0, top = 0.0;
  for (int c = tid; c < a.d; c += 256) {
    const float h = h_at(c);
    sum += (double)h * (double)h;
    top = fmax(top, fabs((double)h * (double)load_as_float(a.weight, c, a.w_f32)));
  }
  sum = wave_sum(sum);
  top = wave_max(top);
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = sum;
    red[1][tid >> 6] = top;
  }
  __syncthreads();
  sum = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
  top = fmax(fmax(red[1][0], red[1][1]), fmax(red[1][2], red[1][3]));
  const double ms = sum / a.d + a.eps;
  const double rstd = ms > 0.0 ? 1.0 / sqrt(ms) : 0.0;
  const float scale = (float)(top * rstd / 127.0);
  const bool empty = scale == 0.0f;
  if (a.out_i8 && tid == 0) a.out_scales[row] = empty ? 1.0f : scale;
  for (int c = tid; c < a.d; c += 256) {
    const float h = h_at(c);
    const double p = (double)h * (double)load_as_float(a.weight, c, a.w_f32);
    if (a.R_out) {  // after h is read: R_out may be R
      if (a.r_f32)
        ((float*)a.R_out)[row * a.ldro + c] = h;
      else
        ((uint16_t*)a.R_out)[row * a.ldro + c] = float_to_bf16_bits(h);
    }
    if (a.out_i8)
      ((int8_t*)a.out)[row * a.ldo + c] = empty ? 0 : (int8_t)(int)rint(127.0 * p / top);
    else
      ((uint16_t*)a.out)[row * a.ldo + c] = float_to_bf16_bits((float)(p * rstd));
  }
}

}  // namespace

hipError_t add_rmsnorm_launch(const void* X, int x_dtype, int64_t ldx, const void* R, int r_dtype,
                              int64_t ldr, void* R_out, int64_t ldro, const void* weight,
                              int w_dtype, double eps, int64_t m, int64_t d, void* out,
                              int out_dtype, int64_t ldo, float* out_scales, hipStream_t stream) {
  NormArgs a;
  a.X = X, a.R = R, a.R_out = R_out, a.weight = weight, a.out = out, a.out_scales = out_scales;
  a.ldx = ldx, a.ldr = ldr, a.ldro = ldro, a.ldo = ldo, a.eps = eps, a.d = (int)d;
  a.x_f32 = x_dtype == GPTQ_F32, a.r_f32 = r_dtype == GPTQ_F32, a.w_f32 = w_dtype == GPTQ_F32;
  a.out_i8 = out_dtype == GPTQ_I8;
  hipLaunchKernelGGL(add_rmsnorm_kernel, dim3((unsigned)m), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace gptq
