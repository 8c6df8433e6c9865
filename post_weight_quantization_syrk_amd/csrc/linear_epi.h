// What a product's sums go through on their way out:
//   y = act(v + bias) + residual,  or, gated, act(v0 + bias0) (v1 + bias1) + residual,
// in float32, rounded once to Y's type.  v0 is the sum of weight row u, v1 that of
// row F + u (the rows of gate and up, one behind the other).
#pragma once

#include "common.h"
#include "kernels.h"

#include <hip/hip_fp16.h>

namespace gptq {

__device__ __forceinline__ bool is_finite(float v) { return v - v == 0.0f; }

// What a sum of the product is made of: rows of X (bf16) and packed weights.
struct Terms {
  const char* x;
  int64_t ldx;  // bytes
  const uint32_t* q;
  const uint16_t *s16, *z16;  // z16 null: symmetric
  int k, ng;
};

// The sum of token t and weight row n, term by term, by a whole wave.
__device__ __forceinline__ float term_by_term(const Terms& a, int lane, int64_t t, int64_t n) {
  float v = 0.0f;
  const uint4* const x = (const uint4*)(a.x + t * a.ldx);
#pragma unroll 1
  for (int w = lane; w < a.k / 8; w += 64) {
    const int64_t g = n * a.ng + 8 * w / (a.k / a.ng);
    const float s = __half2float(__ushort_as_half(a.s16[g]));
    const float z = a.z16 ? __half2float(__ushort_as_half(a.z16[g])) : 8.0f;
    const uint32_t q = a.q[n * (a.k / 8) + w];
    const uint4 u = x[w];
    const uint32_t xs[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v = fmaf(__uint_as_float(xs[j] << 16), s * ((float)((q >> (8 * j)) & 15u) - z), v);
      v = fmaf(__uint_as_float(xs[j] & 0xffff0000u), s * ((float)((q >> (8 * j + 4)) & 15u) - z), v);
    }
  }
  for (int i = 1; i < 64; i *= 2) v += __shfl_xor(v, i);
  return v;
}

__device__ __forceinline__ bool has_nan(const Terms& a, int lane, int64_t t) {
  bool is = false;
  const uint4* const x = (const uint4*)(a.x + t * a.ldx);
#pragma unroll 1
  for (int w = lane; w < a.k / 8; w += 64) {
    const uint4 u = x[w];
    const uint32_t xs[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      is = is || (xs[j] & 0x7fffu) > 0x7f80u || (xs[j] & 0x7fff0000u) > 0x7f800000u;
  }
  return __any(is);
}

// The kernels for few tokens form sum x q and z sum x apart: with an infinity in x, or
// near float32's end, both may be infinite where the sum of x (q - z) is not a NaN.  A
// sum that came out infinite or NaN is therefore formed again, term by term; of a row
// with a NaN it is right as it is.  All lanes of a wave come here; `in`: the lane has a
// sum, v, of token t and weight row n.  (As a function of its own, that is called, it cost
// 64 tokens through 4128 x 4096 in groups of 32 2.4 us of 22.)
__device__ __forceinline__ void right_odd_sums(const Terms& all, bool in, int64_t t, int64_t n, float& v) {
  uint64_t odd = __ballot(in && !is_finite(v));
  if (__builtin_expect(odd == 0, 1)) return;
  // (opaque: else what follows from these is worked out in front, for every call)
  Terms a = all;
  int lane = threadIdx.x & 63;
  asm volatile("" : "+s"(a.k), "+s"(a.ng), "+v"(lane));
  while (odd) {
    const int64_t t1 = __shfl(t, __builtin_ctzll(odd));
    uint64_t same = __ballot(in && t == t1) & odd;
    odd &= ~same;
    if (has_nan(a, lane, t1)) continue;
    for (; same; same &= same - 1) {
      const int l = __builtin_ctzll(same);
      const float right = term_by_term(a, lane, t1, __shfl(n, l));
      if (lane == l) v = right;
    }
  }
}

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
// Terms without weights: the sums are right as they are.
template <bool GATED>
__global__ __launch_bounds__(256) void join_finish_kernel(const float* __restrict__ part, int64_t m,
                                                          int n, int splits, Epilogue e, Terms terms) {
  const int chunks = (e.F + 255) / 256;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), row = t / chunks;
  const int u = 256 * (int)(t - row * chunks) + (threadIdx.x & 63);
  const int cols = min(4, (e.F - u + 63) / 64);
  if (row >= m) return;
  float v0[4] = {}, v1[4] = {};
  if (cols > 0) {
    const float* p = part + row * n + u;
    const int64_t next = m * n;
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
  }
  float odd = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) odd = fmaf(v0[k], 0.0f, fmaf(v1[k], 0.0f, odd));
  if (terms.q && __builtin_expect(__any(odd != 0.0f), 0)) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      right_odd_sums(terms, k < cols, row, u + 64 * k, v0[k]);
      if constexpr (GATED) right_odd_sums(terms, k < cols, row, e.F + u + 64 * k, v1[k]);
    }
  }
  if (cols > 0) finish4<GATED, 64>(e, row, u, cols, v0, v1);
}

template <bool GATED>
hipError_t join_finish_launch(const float* part, int64_t m, int n, int splits, const Epilogue& e,
                              const Terms& terms, hipStream_t stream) {
  hipLaunchKernelGGL((join_finish_kernel<GATED>), dim3((unsigned)ceil_div(m * ((e.F + 255) / 256), 4)),
                     dim3(256), 0, stream, part, m, n, splits, e, terms);
  return hipGetLastError();
}

}  // namespace gptq
