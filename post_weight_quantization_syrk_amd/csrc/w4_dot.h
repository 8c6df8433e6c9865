// The products of packed 4-bit weights with one token: bf16 or int8 activations,
// one kernel template for both.
//   Y[n] = sx sum_g s[n][g] (sum_{k in g} x q - z[n][g] sum_{k in g} x)
//
// A wave keeps a run of 2048 k of X in registers, 32 consecutive k per lane,
// and takes that run of one weight row after the other: 1 KB of a row per
// load, 16 bytes per lane.  A lane's 32 codes lie in one group, so its sum of
// x q is finished with the lane's own scale and zero and sum of x, and what is
// added over lanes, and over the waves that share a row, are final terms.
//
// Bound by reading the weights: 28672 x 8192, one scale per row, takes 24 us
// (4.9 TB/s, what a large copy reaches; the norm's kernel, which writes half of
// its bytes, reaches 5.9).  Dot-product instructions, two bf16 or
// four int8 terms each, keep the vector units below that; matrix instructions
// would do sixteen tokens' work for one, and their operands' layout spreads a
// load over sixteen rows.  4096 x 4096 in groups of 128 takes 3.8 us, of which
// an empty launch is 2.6.
#pragma once

#include "w4_vec.h"

namespace gptq {
namespace w4vec {

__device__ __forceinline__ float dot2(bf16x2 a, bf16x2 b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(a, b, c, false);
}
__device__ __forceinline__ bf16x2 as_bf16x2(uint32_t u) {
  bf16x2 v;
  __builtin_memcpy(&v, &u, 4);
  return v;
}

// Sum of v over the 16 lanes of each row of lanes, in every lane.
__device__ __forceinline__ float row_sum(float v) {
  auto add = [&](auto ctrl) __attribute__((always_inline)) {
    v += __int_as_float(
        __builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  add(std::integral_constant<int, 0x128>());  // row_ror:8, 4, 2, 1
  add(std::integral_constant<int, 0x124>());
  add(std::integral_constant<int, 0x122>());
  add(std::integral_constant<int, 0x121>());
  return v;
}

// Sums of four values over the wave: lane row r (of 16 lanes) gets the sum of
// value 0, 2, 1, 3 for r = 0, 1, 2, 3.  Each swap folds two registers into one.
__device__ __forceinline__ float wave_sum4(const float v[4]) {
  auto fold32 = [](float a, float b) __attribute__((always_inline)) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  const float p = fold32(v[0], v[1]), q = fold32(v[2], v[3]);
  const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(p), __float_as_uint(q), false, false);
  return row_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// ks: waves that share a row (runs per row); rpw: rows per wave, a
// multiple of 4.
template <bool I8, class E>
__global__ __launch_bounds__(1024) void w4_dot_kernel(VecArgs a, int G, int ks, int rpw, E epi) {
  extern __shared__ float red[];  // [rows of the workgroup][ks]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int seg = wave % ks, rg = wave / ks, rows = (int)(blockDim.x >> 6) / ks * rpw;
  const int64_t n0 = (int64_t)blockIdx.x * rows + rg * rpw;
  // gated: even rows are gate rows, odd ones the up rows that go with them
  auto valid_row = [&](int64_t n) __attribute__((always_inline)) {
    if constexpr (E::gated)
      return min(n >> 1, (int64_t)epi.e.F - 1) + (n & 1) * epi.e.F;
    else
      return min(n, (int64_t)a.n - 1);
  };
  const int row_bytes = a.k / 2;
  const int k0 = seg * RUN + 32 * lane;
  const bool in = k0 < a.k;
  const int kc = in ? k0 : 0;  // lanes past the row's end: x = 0
  const int g = kc / G;

  struct Rows {
    uint4 w[4];
    uint16_t s[4], z[4];
  };
  auto load = [&](int r, Rows& v) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t n = valid_row(n0 + r + u);
      v.w[u] = *(const uint4*)((const char*)a.q + n * row_bytes + kc / 2);
      v.s[u] = a.s16[n * a.ng + g];
      v.z[u] = a.z16 ? a.z16[n * a.ng + g] : (uint16_t)0x4800;  // 8
    }
  };
  Rows cur, nxt;
  load(0, cur);

  // x in the order in which a word's codes come apart: 0 2 4 6 1 3 5 7
  uint32_t x[I8 ? 8 : 16];
  float xsum = 0.0f;
  int xsumi = 0;
  const uint4* p = (const uint4*)(a.x + kc * (I8 ? 1 : 2));
#pragma unroll
  for (int j = 0; j < (I8 ? 2 : 4); ++j) {
    uint4 v = p[j];
    if (!in) v = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (I8) {
      x[4 * j] = __builtin_amdgcn_perm(v.y, v.x, 0x06040200u);
      x[4 * j + 1] = __builtin_amdgcn_perm(v.y, v.x, 0x07050301u);
      x[4 * j + 2] = __builtin_amdgcn_perm(v.w, v.z, 0x06040200u);
      x[4 * j + 3] = __builtin_amdgcn_perm(v.w, v.z, 0x07050301u);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        xsumi = __builtin_amdgcn_sdot4((int)x[4 * j + e], 0x01010101, xsumi, false);
    } else {
      x[4 * j] = __builtin_amdgcn_perm(v.y, v.x, 0x05040100u);
      x[4 * j + 1] = __builtin_amdgcn_perm(v.w, v.z, 0x05040100u);
      x[4 * j + 2] = __builtin_amdgcn_perm(v.y, v.x, 0x07060302u);
      x[4 * j + 3] = __builtin_amdgcn_perm(v.w, v.z, 0x07060302u);
      const bf16x2 ones = as_bf16x2(0x3f803f80u);
#pragma unroll
      for (int e = 0; e < 4; ++e) xsum = dot2(as_bf16x2(x[4 * j + e]), ones, xsum);
    }
  }

  for (int r = 0; r < rpw; r += 4) {
    if (r + 4 < rpw) load(r + 4, nxt);
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t w[4] = {cur.w[u].x, cur.w[u].y, cur.w[u].z, cur.w[u].w};
      const float s = half_bits(cur.s[u]);
      if constexpr (I8) {
        int acc = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc = __builtin_amdgcn_sdot4((int)x[2 * j], (int)(w[j] & 0x0f0f0f0fu), acc, false);
          acc = __builtin_amdgcn_sdot4((int)x[2 * j + 1], (int)((w[j] >> 4) & 0x0f0f0f0fu), acc,
                                       false);
        }
        v[u] = s * (float)(acc - __mul24(whole_zero(cur.z[u]), xsumi));
      } else {
        float acc = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t ev = w[j] & 0x0f0f0f0fu, od = (w[j] >> 4) & 0x0f0f0f0fu;
          const bf16x2 b0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(ev, 512.0f, false);
          const bf16x2 b1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(ev, 512.0f, true);
          const bf16x2 b2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(od, 512.0f, false);
          const bf16x2 b3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(od, 512.0f, true);
          acc = dot2(as_bf16x2(x[4 * j]), b0, acc);
          acc = dot2(as_bf16x2(x[4 * j + 1]), b1, acc);
          acc = dot2(as_bf16x2(x[4 * j + 2]), b2, acc);
          acc = dot2(as_bf16x2(x[4 * j + 3]), b3, acc);
        }
        v[u] = s * fmaf(-half_bits(cur.z[u]), xsum, acc);
      }
    }
    const float sum = wave_sum4(v);
    const int lr = lane >> 4, u = ((lr & 1) << 1) | (lr >> 1);
    if ((lane & 15) == 0) red[(rg * rpw + r + u) * ks + seg] = sum;
    cur = nxt;
  }
  __syncthreads();
  auto summed = [&](int row) __attribute__((always_inline)) {
    float v = 0.0f;
    for (int s = 0; s < ks; ++s) v += red[row * ks + s];
    return v;
  };
  // whole waves go round; sums that are not finite in a second one
  const int first = threadIdx.x & ~63;
  auto finished = [&](auto second) __attribute__((always_inline)) {
    constexpr bool SECOND = decltype(second)::value;
    bool odd = false;
    if constexpr (E::gated) {
      for (int p0 = first; p0 < rows / 2; p0 += blockDim.x) {
        const int p = p0 + lane;
        const int64_t u = (int64_t)blockIdx.x * (rows / 2) + p;
        bool now = p < rows / 2 && u < epi.e.F;
        float v0 = now ? summed(2 * p) : 0.0f, v1 = now ? summed(2 * p + 1) : 0.0f;
        const bool fin = is_finite(v0) && is_finite(v1);
        odd = odd || !fin;
        now = now && fin != SECOND;
        if constexpr (SECOND) {
          right_odd_sums(terms_of(a), now, 0, u, v0);
          right_odd_sums(terms_of(a), now, 0, epi.e.F + u, v1);
        }
        if (now) finish<true>(epi.e, 0, u, v0, v1);
      }
    } else if constexpr (E::linear) {
      for (int row0 = first; row0 < rows; row0 += blockDim.x) {
        const int row = row0 + lane;
        const int64_t n = (int64_t)blockIdx.x * rows + row;
        bool now = row < rows && n < a.n;
        float v = now ? summed(row) : 0.0f;
        const bool fin = is_finite(v);
        odd = odd || !fin;
        now = now && fin != SECOND;
        if constexpr (SECOND) right_odd_sums(terms_of(a), now, 0, n, v);
        if (now) finish<false>(epi.e, 0, n, v, 0.0f);
      }
    }
    return __any(odd);
  };
  if constexpr (E::linear) {
    if (__builtin_expect(finished(std::false_type()), 0)) finished(std::true_type());
    return;
  }
  for (int row = threadIdx.x; row < rows; row += blockDim.x) {
    const int64_t n = (int64_t)blockIdx.x * rows + row;
    float v = summed(row);
    if constexpr (I8) v *= a.sx[0];
    if (n < a.n) a.y[n] = v;
  }
}

// Rows per wave: few enough that the launch has some 8192 waves' rows at once.
template <bool I8, class E = Plain>
hipError_t dot_launch(const VecArgs& a, int G, hipStream_t stream, const E& e = E{}) {
  const int ks = (int)ceil_div(a.k, RUN), rgs = ks >= 8 ? 1 : 8 / ks;
  int rpw = 4;
  while (rpw < 32 && (int64_t)a.n * ks / rpw > 8192) rpw *= 2;
  const int rows = rgs * rpw;
  hipLaunchKernelGGL((w4_dot_kernel<I8, E>), dim3((unsigned)ceil_div(a.n, rows)), dim3(64 * ks * rgs),
                     (size_t)rows * ks * sizeof(float), stream, a, G == 0 ? a.k : G, ks, rpw, e);
  return hipGetLastError();
}

}  // namespace w4vec
}  // namespace gptq
