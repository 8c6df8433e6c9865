// What a product's sums go through on their way out:
//   y = act(v + bias) + residual,  or, gated, act(v0 + bias0) (v1 + bias1) + residual,
// in float32, rounded once to Y's type.  v0 is the sum of weight row u, v1 that of
// row F + u (the rows of gate and up, one behind the other).
#pragma once

#include "common.h"
#include "kernels.h"

namespace gptq {

__device__ __forceinline__ float load_as_float(const void* p, int64_t i, bool f32) {
  return f32 ? ((const float*)p)[i] : bf16_bits_to_float(((const uint16_t*)p)[i]);
}

// GELU by its tanh form is v times the logistic function of twice the tanh's
// argument; with 1 + tanh it would lose the lower tail to cancellation, as GELU
// would with 1 + erf.
__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {
    case ACT_RELU: return v > 0.0f ? v : v != v ? v : 0.0f;
    case ACT_SILU: return v / (1.0f + expf(-v));
    case ACT_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    case ACT_GELU_TANH: {
      const float u = 1.5957691216057308f * fmaf(0.044715f * v * v, v, v);
      return v / (1.0f + expf(-u));
    }
    default: return v;
  }
}

// Stores the output of row `row`, column u; v1 is not read unless GATED.
template <bool GATED>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t row, int64_t u, float v0,
                                       float v1) {
  if (e.bias) {
    v0 += load_as_float(e.bias, u, e.bias_f32);
    if constexpr (GATED) v1 += load_as_float(e.bias, e.F + u, e.bias_f32);
  }
  float y = activate(e.act, v0);
  if constexpr (GATED) y *= v1;
  if (e.res) y += load_as_float(e.res, row * e.ldr + u, e.res_f32);
  if (e.y_f32)
    ((float*)e.y)[row * e.ldy + u] = y;
  else
    ((__bf16*)e.y)[row * e.ldy + u] = (__bf16)y;
}

// Up to four outputs of a row, STEP columns apart, n of which are there.
template <bool GATED, int STEP = 1>
__device__ __forceinline__ void finish4(const Epilogue& e, int64_t row, int64_t u, int n, float v0[4],
                                        float v1[4]) {
  if (e.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = u + STEP * min(i, n - 1);
      v0[i] += load_as_float(e.bias, c, e.bias_f32);
      if constexpr (GATED) v1[i] += load_as_float(e.bias, e.F + c, e.bias_f32);
    }
  }
  float res[4] = {};
  if (e.res) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      res[i] = load_as_float(e.res, row * e.ldr + u + STEP * min(i, n - 1), e.res_f32);
  }
  if (e.act != ACT_NONE) {
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {  // (one copy of the activations: the values go round)
      const float t = activate(e.act, v0[0]);
      v0[0] = v0[1], v0[1] = v0[2], v0[2] = v0[3], v0[3] = t;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (GATED) v0[i] *= v1[i];
    v0[i] += res[i];
  }
  const int64_t at = row * e.ldy + u;
  if (STEP == 1 && e.vec4 && n == 4) {
    if (e.y_f32) {
      *(float4*)((float*)e.y + at) = make_float4(v0[0], v0[1], v0[2], v0[3]);
    } else {
      typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
      *(bf16x4*)((__bf16*)e.y + at) =
          bf16x4{(__bf16)v0[0], (__bf16)v0[1], (__bf16)v0[2], (__bf16)v0[3]};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= n) break;
    if (e.y_f32)
      ((float*)e.y)[at + STEP * i] = v0[i];
    else
      ((__bf16*)e.y)[at + STEP * i] = (__bf16)v0[i];
  }
}

// The splits' sums [splits][m][n] added in split order, then finished: a wave takes
// 256 columns of a row, a lane four of them 64 apart, so that every load and store
// is of neighbours whatever n's alignment; four splits' loads are in flight at a time.
template <bool GATED>
__global__ __launch_bounds__(256) void join_finish_kernel(const float* __restrict__ part, int64_t m,
                                                          int n, int splits, Epilogue e) {
  const int chunks = (e.F + 255) / 256;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), row = t / chunks;
  const int u = 256 * (int)(t - row * chunks) + (threadIdx.x & 63);
  const int cols = min(4, (e.F - u + 63) / 64);
  if (row >= m || cols <= 0) return;
  const float* p = part + row * n + u;
  const int64_t next = m * n;
  float v0[4] = {}, v1[4] = {};
  for (int s = 0; s < splits; s += 4) {
    float a[4][4], b[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* q = p + min(s + i, splits - 1) * next;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[i][k] = q[64 * min(k, cols - 1)];
        if constexpr (GATED) b[i][k] = q[e.F + 64 * min(k, cols - 1)];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s + i >= splits) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v0[k] += a[i][k];
        if constexpr (GATED) v1[k] += b[i][k];
      }
    }
  }
  finish4<GATED, 64>(e, row, u, cols, v0, v1);
}

template <bool GATED>
hipError_t join_finish_launch(const float* part, int64_t m, int n, int splits, const Epilogue& e,
                              hipStream_t stream) {
  hipLaunchKernelGGL((join_finish_kernel<GATED>), dim3((unsigned)ceil_div(m * ((e.F + 255) / 256), 4)),
                     dim3(256), 0, stream, part, m, n, splits, e);
  return hipGetLastError();
}

}  // namespace gptq
