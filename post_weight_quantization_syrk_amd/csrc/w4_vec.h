// The products of packed 4-bit weights with a few tokens (m <= 64): bf16 or
// int8 activations, one kernel template for both.
//   Y[i][n] = sx[i] sum_g s[n][g] (sum_{k in g} x q - z[n][g] sum_{k in g} x)
//
// A workgroup owns 16 R weight rows and all tokens; its waves take 256-byte
// runs of k in turn and their sums meet in LDS at the end, in wave order.
// Weights go from memory to registers, 16 bytes per lane: lane l holds 32
// consecutive codes of row l % 16, and the four lanes of a row 64 bytes.
// A matrix instruction wants, in lane quarter h, the h-th piece of one run of
// k.  With groups of 128 (or one per row) the order of k inside a chunk is
// free, so word j of every lane makes up instruction j; with groups of 32 or
// 64 a 4 x 4 transposition of words between the quarters (four swaps for 32
// codes) puts consecutive words side by side first.
// The zero is not taken off the codes: x q and x are summed apart (the sum of
// x by the same instruction against ones, shared by all rows), and joined per
// group.
#pragma once

#include "common.h"

#include <hip/hip_fp16.h>

namespace gptq {
namespace w4vec {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

constexpr int KCH = 128;
constexpr int max_waves(int nt) { return nt == 1 ? 16 : 8; }

struct VecArgs {
  const char* x;        // rows of X
  const float* sx;      // x_scales (int8 X)
  const uint32_t* q;
  const uint16_t* s16;
  const uint16_t* z16;  // null: symmetric
  float* y;
  int64_t ldx;          // bytes
  int m, n, k, ng;
};

template <bool I8>
struct Types;
template <>
struct Types<false> {
  typedef f32x4 acc_t;
};
template <>
struct Types<true> {
  typedef i32x4 acc_t;
};

// word j of lane quarter h <-> word h of lane quarter j
__device__ __forceinline__ void transpose4(uint32_t w[4]) {
  u32x2 a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  u32x2 b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  u32x2 lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  u32x2 hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w[0] = lo[0], w[1] = lo[1], w[2] = hi[0], w[3] = hi[1];
}

// The codes of a word as bytes in their order.
__device__ __forceinline__ uint2 code_bytes(uint32_t w) {
  const uint32_t ev = w & 0x0f0f0f0fu, od = (w >> 4) & 0x0f0f0f0fu;
  return make_uint2(__builtin_amdgcn_perm(od, ev, 0x05010400u),
                    __builtin_amdgcn_perm(od, ev, 0x07030602u));
}

// The codes of a word as bf16.  As an 8-bit float with four exponent and three
// mantissa bits the byte 0000 cccc is c 2^-9 (below 8 a subnormal, from 8 the
// first binade, with the same step), so one conversion scaled by 2^9 turns two
// bytes into two bf16, exactly.
__device__ __forceinline__ bf16x8 code_bf16(uint32_t w) {
  const uint2 b = code_bytes(w);
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.x, 512.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.x, 512.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.y, 512.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.y, 512.0f, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ float half_bits(uint16_t b) {
  return __half2float(__ushort_as_half(b));
}

// I8: int8 X; NT: tiles of 16 tokens; R: tiles of 16 weight rows; G: group
// size, 0 for one group per row; CPS: chunks of 128 k per step of a wave.
template <bool I8, int NT, int R, int G, int CPS>
__global__ __launch_bounds__(64 * max_waves(NT)) void w4_vec_kernel(VecArgs a) {
  typedef typename Types<I8>::acc_t acc_t;
  constexpr bool TR = G == 32 || G == 64;
  constexpr int GPC = G == 0 ? 1 : KCH / G;          // groups per chunk
  constexpr int XB = I8 ? 1 : 2;                     // bytes of an X element
  extern __shared__ float red[];                     // [waves][R * NT * 4][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int l16 = lane & 15, h = lane >> 4;
  const int n0 = blockIdx.x * 16 * R;
  const int row_bytes = a.k / 2;
  const int nst = (a.k + CPS * KCH - 1) / (CPS * KCH);

  const char* qrow[R];
  int64_t srow[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t n = min(n0 + 16 * r + l16, a.n - 1);
    qrow[r] = (const char*)a.q + n * row_bytes;
    srow[r] = n * a.ng;
  }
  const char* xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = a.x + (int64_t)min(16 * t + l16, a.m - 1) * a.ldx;

  struct Step {
    uint4 w[CPS][R];
    uint32_t x[CPS][NT][I8 ? 8 : 16];  // 32 k of one token: four 8-k pieces
    uint16_t s[CPS][R][GPC], z[CPS][R][GPC];
  };
  auto load = [&](int st, Step& v) __attribute__((always_inline)) {
#pragma unroll
    for (int cc = 0; cc < CPS; ++cc) {
      const int c = st * CPS + cc;
#pragma unroll
      for (int r = 0; r < R; ++r)
        v.w[cc][r] = *(const uint4*)(qrow[r] + min(c * (KCH / 2) + 16 * h, row_bytes - 16));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (TR) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = min(c * KCH + 32 * j + 8 * h, a.k - 8);
            if constexpr (I8) {
              const uint2 p = *(const uint2*)(xrow[t] + k);
              v.x[cc][t][2 * j] = p.x, v.x[cc][t][2 * j + 1] = p.y;
            } else {
              const uint4 p = *(const uint4*)(xrow[t] + 2 * k);
              v.x[cc][t][4 * j] = p.x, v.x[cc][t][4 * j + 1] = p.y;
              v.x[cc][t][4 * j + 2] = p.z, v.x[cc][t][4 * j + 3] = p.w;
            }
          }
        } else {
          const char* p = xrow[t] + XB * min(c * KCH + 32 * h, a.k - 32);
#pragma unroll
          for (int j = 0; j < 2 * XB; ++j) {
            const uint4 u = *(const uint4*)(p + 16 * j);
            v.x[cc][t][4 * j] = u.x, v.x[cc][t][4 * j + 1] = u.y;
            v.x[cc][t][4 * j + 2] = u.z, v.x[cc][t][4 * j + 3] = u.w;
          }
        }
      }
      if constexpr (G != 0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int g = 0; g < GPC; ++g) {
            const int64_t i = srow[r] + min(c * GPC + g, a.ng - 1);
            v.s[cc][r][g] = a.s16[i];
            v.z[cc][r][g] = a.z16 ? a.z16[i] : (uint16_t)0x4800;  // 8
          }
      }
    }
  };

  float tot[R][NT][4];
  acc_t acc0[R][NT], one0[NT];  // G == 0: over the whole row
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    one0[t] = acc_t{0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      acc0[r][t] = acc_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[r][t][i] = 0.0f;
    }
  }
  // tot += s (acc - z one)
  auto join = [&](float t, float s, uint16_t zb, auto acc, auto one) __attribute__((always_inline)) {
    if constexpr (I8) {
      const int z = (int)fminf(fmaxf(rintf(half_bits(zb)), -100.0f), 100.0f);
      return fmaf(s, (float)(acc - __mul24(z, one)), t);
    } else {
      return fmaf(s, fmaf(-half_bits(zb), one, acc), t);
    }
  };

  auto compute = [&](int st, Step& v) __attribute__((always_inline)) {
#pragma unroll
    for (int cc = 0; cc < CPS; ++cc) {
      const int c = st * CPS + cc;
      // pieces past the row's end count as zeros
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = c * KCH + 32 * (TR ? j : h) < a.k;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < (I8 ? 2 : 4); ++e)
            v.x[cc][t][(I8 ? 2 : 4) * j + e] = in ? v.x[cc][t][(I8 ? 2 : 4) * j + e] : 0u;
      }
      uint32_t w[R][4];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        w[r][0] = v.w[cc][r].x, w[r][1] = v.w[cc][r].y, w[r][2] = v.w[cc][r].z,
        w[r][3] = v.w[cc][r].w;
        if constexpr (TR) transpose4(w[r]);
      }
      if constexpr (!I8) {
        bf16x8 b[R][4];
        const __bf16 o = (__bf16)1.0f;
        const bf16x8 ones = {o, o, o, o, o, o, o, o};
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) b[r][j] = code_bf16(w[r][j]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          bf16x8 x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) __builtin_memcpy(&x[j], &v.x[cc][t][4 * j], 16);
#pragma unroll
          for (int g = 0; g < GPC; ++g) {
            acc_t one = {0, 0, 0, 0}, acc[R];
            if constexpr (G == 0) one = one0[t];
#pragma unroll
            for (int r = 0; r < R; ++r) {
              acc[r] = acc_t{0, 0, 0, 0};
              if constexpr (G == 0) acc[r] = acc0[r][t];
            }
#pragma unroll
            for (int j = 4 * g / GPC; j < 4 * (g + 1) / GPC; ++j) {
              one = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j], ones, one, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < R; ++r)
                acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j], b[r][j], acc[r], 0, 0, 0);
            }
            if constexpr (G == 0) one0[t] = one;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              if constexpr (G == 0) {
                acc0[r][t] = acc[r];
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  tot[r][t][i] = join(tot[r][t][i], half_bits(v.s[cc][r][g]), v.z[cc][r][g],
                                      acc[r][i], one[i]);
              }
            }
          }
        }
      } else {
        uint2 b[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) b[r][j] = code_bytes(w[r][j]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t* x = v.x[cc][t];
#pragma unroll
          for (int g = 0; g < GPC; ++g) {
            acc_t one = {0, 0, 0, 0}, acc[R];
            if constexpr (G == 0) one = one0[t];
#pragma unroll
            for (int r = 0; r < R; ++r) {
              acc[r] = acc_t{0, 0, 0, 0};
              if constexpr (G == 0) acc[r] = acc0[r][t];
            }
            if constexpr (G == 32) {
              auto two = [](uint32_t lo, uint32_t hi) { return (long)(((uint64_t)hi << 32) | lo); };
              const long xv = two(x[2 * g], x[2 * g + 1]);
              one = __builtin_amdgcn_mfma_i32_16x16x32_i8(xv, 0x0101010101010101l, one, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < R; ++r)
                acc[r] = __builtin_amdgcn_mfma_i32_16x16x32_i8(xv, two(b[r][g].x, b[r][g].y),
                                                               acc[r], 0, 0, 0);
            } else {
              const int o = 0x01010101;
#pragma unroll
              for (int j = 2 * g / GPC; j < 2 * (g + 1) / GPC; ++j) {
                const i32x4 xv = {(int)x[4 * j], (int)x[4 * j + 1], (int)x[4 * j + 2],
                                  (int)x[4 * j + 3]};
                one = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv, i32x4{o, o, o, o}, one, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                  const i32x4 bv = {(int)b[r][2 * j].x, (int)b[r][2 * j].y,
                                    (int)b[r][2 * j + 1].x, (int)b[r][2 * j + 1].y};
                  acc[r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv, bv, acc[r], 0, 0, 0);
                }
              }
            }
            if constexpr (G == 0) one0[t] = one;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              if constexpr (G == 0) {
                acc0[r][t] = acc[r];
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  tot[r][t][i] = join(tot[r][t][i], half_bits(v.s[cc][r][g]), v.z[cc][r][g],
                                      acc[r][i], one[i]);
              }
            }
          }
        }
      }
    }
  };

  Step cur, nxt;
  if (wave < nst) load(wave, cur);
  for (int st = wave; st < nst; st += waves) {
    if (st + waves < nst) load(st + waves, nxt);
    compute(st, cur);
    cur = nxt;
  }
  if constexpr (G == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float s = half_bits(a.s16[srow[r]]);
      const uint16_t z = a.z16 ? a.z16[srow[r]] : (uint16_t)0x4800;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[r][t][i] = join(0.0f, s, z, acc0[r][t][i], one0[t][i]);
    }
  }
  constexpr int PER = R * NT * 4;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(wave * PER + (r * NT + t) * 4 + i) * 64 + lane] = tot[r][t][i];
  __syncthreads();
  for (int e = wave; e < PER; e += waves) {
    float v = 0.0f;
    for (int w = 0; w < waves; ++w) v += red[(w * PER + e) * 64 + lane];
    const int i = e & 3, t = (e >> 2) % NT, r = (e >> 2) / NT;
    const int token = 16 * t + 4 * h + i, n = n0 + 16 * r + l16;
    if (token < a.m && n < a.n) {
      if constexpr (I8) v *= a.sx[token];
      a.y[(int64_t)token * a.n + n] = v;
    }
  }
}

// Waves per workgroup: enough of them over the whole launch to keep the memory
// busy, no more than there are steps.
inline int vec_waves(int64_t groups, int steps, int most) {
  int w = 4;
  while (w < most && groups * w < 4096) w *= 2;
  while (w > 1 && w > steps) w /= 2;
  return w;
}

template <bool I8, int NT, int R, int G>
hipError_t vec_launch_one(const VecArgs& a, hipStream_t stream) {
  constexpr int CPS = NT == 1 && (I8 || G == 0 || G == 128) ? 2 : 1;
  const int64_t groups = ceil_div(a.n, 16 * R);
  const int waves = vec_waves(groups, (int)ceil_div(a.k, CPS * KCH), max_waves(NT));
  const size_t lds = (size_t)waves * R * NT * 4 * 64 * sizeof(float);
  hipLaunchKernelGGL((w4_vec_kernel<I8, NT, R, G, CPS>), dim3((unsigned)groups), dim3(64 * waves),
                     lds, stream, a);
  return hipGetLastError();
}

template <bool I8, int NT, int R>
hipError_t vec_launch_g(const VecArgs& a, int G, hipStream_t stream) {
  switch (G) {
    case 32: return vec_launch_one<I8, NT, R, 32>(a, stream);
    case 64: return vec_launch_one<I8, NT, R, 64>(a, stream);
    case 128: return vec_launch_one<I8, NT, R, 128>(a, stream);
    default: return vec_launch_one<I8, NT, R, 0>(a, stream);
  }
}

template <bool I8>
hipError_t vec_launch(const VecArgs& a, int G, hipStream_t stream) {
  if (a.m <= 16) return vec_launch_g<I8, 1, 1>(a, G, stream);
  if (a.m <= 32) return vec_launch_g<I8, 2, 1>(a, G, stream);
  return vec_launch_g<I8, 4, 1>(a, G, stream);
}

}  // namespace w4vec
}  // namespace gptq
