// Residual addition, root-mean-square norm, and an output in bf16 or in 8 bits
// with a scale per row:
//   h = x + r (fp32, rounded to r's type),  y_c = h_c w_c / sqrt(mean h^2 + eps)
//   8 bits: p_c = h_c w_c, P = max |p_c|, q_c = rint(127 p_c / P),
//           scale = P / sqrt(mean h^2 + eps) / 127
// The norm's own factor cancels in the codes, so they depend on no sum's
// order; p is exact in float64 and the quotient is formed there.
//
// Bound by memory.  A workgroup holds a row of up to 16384 in registers between
// the one reduction (of sum h^2 and max |p|, together) and the output: x and r
// are read once, h and the output written once.  (Longer rows are read twice, in
// the same launch.)  The reductions are in float64: its operations run at the
// rate of float32 ones here, and squares neither overflow nor vanish.  The
// vector units come next (57% busy at 16384 x 8192 with bf16 output): divisions
// are done as reciprocals with an iteration, and a code takes six operations
// (4096 x 4096 to 8 bits, 31.6 us with divisions, rounding and conversions as
// such, 27.5 so).
// Measured, residual and all, GPU time per call in a replayed graph: 16384 x
// 8192 bf16 181 us (5.9 TB/s; a large copy reaches 4.9), in 8 bits 165 (5.7);
// 4096 x 4096 in 8 bits 27.5 (4.3); 1000 x 5003 float32, unaligned rows, 14.3
// (4.5); one row of 4096 3.5, a launch.
#include "common.h"
#include "kernels.h"

#include "../../include/gptq.h"

namespace gptq {

namespace {

struct NormArgs {
  const char* x;
  const char* r;
  char* r_out;
  const char* w;
  char* out;
  float* scales;
  int64_t ldx, ldr, ldro, ldo;  // elements
  double eps, inv_d;
  int d;
  int out_i8;
};

constexpr int REG_D = 16384;  // longest row held in registers

enum Kind { NONE, BF16, F32 };

__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const __bf16 b = (__bf16)f;  // nearest, ties to even
  uint16_t u;
  __builtin_memcpy(&u, &b, 2);
  return u;
}

// v combined with a copy of itself whose lanes are moved by a DPP control.
template <int CTRL, class F>
__device__ __forceinline__ double dpp_fold(double v, F f) {
  const int lo = __builtin_amdgcn_mov_dpp(__double2loint(v), CTRL, 0xF, 0xF, false);
  const int hi = __builtin_amdgcn_mov_dpp(__double2hiint(v), CTRL, 0xF, 0xF, false);
  return f(v, __hiloint2double(hi, lo));
}

// f over the wave, in every lane.
template <class F>
__device__ __forceinline__ double wave_fold(double v, F f) {
  v = dpp_fold<0x128>(v, f);  // row_ror:8, 4, 2, 1: over 16 lanes
  v = dpp_fold<0x124>(v, f);
  v = dpp_fold<0x122>(v, f);
  v = dpp_fold<0x121>(v, f);
  const auto lo16 = __builtin_amdgcn_permlane16_swap(__double2loint(v), __double2loint(v), false, false);
  const auto hi16 = __builtin_amdgcn_permlane16_swap(__double2hiint(v), __double2hiint(v), false, false);
  v = f(__hiloint2double(hi16[0], lo16[0]), __hiloint2double(hi16[1], lo16[1]));
  const auto lo32 = __builtin_amdgcn_permlane32_swap(__double2loint(v), __double2loint(v), false, false);
  const auto hi32 = __builtin_amdgcn_permlane32_swap(__double2hiint(v), __double2hiint(v), false, false);
  return f(__hiloint2double(hi32[0], lo32[0]), __hiloint2double(hi32[1], lo32[1]));
}

// 1 / x in float64: the instruction's estimate (at least 22 bits) and one
// iteration, which doubles them.  x in the range of 127 / x's use.
__device__ __forceinline__ double reciprocal(double x) {
  const double r = __builtin_amdgcn_rcp(x);
  return fma(r, fma(-x, r, 1.0), r);
}

// 1 / sqrt(x) of a positive number, with an iteration of third order: to the
// last bits of a float64.
__device__ __forceinline__ double reciprocal_root(double x) {
  double r = __builtin_amdgcn_rsq(x);
  const double e = fma(-x * r, r, 1.0);
  return fma(r * e, fma(e, 0.375, 0.5), r);
}

// Sum of `sum` and maximum of `top` over the workgroup, in every thread; the
// waves' parts are joined in wave order.
__device__ __forceinline__ void fold_row(double& sum, double& top, double (*red)[16]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = (int)blockDim.x >> 6;
  sum = wave_fold(sum, [](double p, double q) { return p + q; });
  top = wave_fold(top, [](double p, double q) { return fmax(p, q); });
  if (waves > 1) {
    if (lane == 0) red[0][wave] = sum, red[1][wave] = top;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < waves; i += 4) {  // four at a time, read together
      double p[4], q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = red[0][i + j], q[j] = red[1][i + j];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum += i + j < waves ? p[j] : 0.0;
        top = fmax(top, i + j < waves ? q[j] : 0.0);
      }
    }
  }
}

// Eight consecutive elements of a row as they are in memory.
template <Kind K>
struct Raw {
  uint32_t u[K == F32 ? 8 : 4];
};

// Pieces at an address that only the elements' own size divides: global loads
// and stores take those (4096 x 5003 bf16 to 8 bits: 43 us; 95 by elements, one
// per lane; 4096 x 5000, aligned: 35).
typedef uint32_t any_u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t any_u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t any_u32x2_4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t any_u32x2_2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t any_u32x2_1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t any_u32_2 __attribute__((aligned(2)));
typedef uint32_t any_u32_1 __attribute__((aligned(1)));
typedef uint16_t any_u16_1 __attribute__((aligned(1)));

// Elements c .. c + 7 of a row of d.  VEC: the row starts on 16 bytes and d is
// whole eights; otherwise any address, and the row's last piece by elements.
template <Kind K, bool VEC>
__device__ __forceinline__ void load8(const char* row, int c, int d, Raw<K>& o) {
  if constexpr (VEC) {
    const uint4* p = (const uint4*)(row + (int64_t)(c < d ? c : 0) * (K == F32 ? 4 : 2));
    const uint4 a = p[0];
    o.u[0] = a.x, o.u[1] = a.y, o.u[2] = a.z, o.u[3] = a.w;
    if constexpr (K == F32) {
      const uint4 b = p[1];
      o.u[4] = b.x, o.u[5] = b.y, o.u[6] = b.z, o.u[7] = b.w;
    }
  } else if ((int)__builtin_amdgcn_readfirstlane(c) >= d) {  // a wave past the row
#pragma unroll
    for (int e = 0; e < (K == F32 ? 8 : 4); ++e) o.u[e] = 0u;
  } else if (d >= 8) {
    // the last piece from the row's last eight, moved down: what does not belong
    // to it (and may be written by others meanwhile) falls out
    const int at = min(c, d - 8), by = c - at;
    if constexpr (K == F32) {
      const any_u32x4_4* p = (const any_u32x4_4*)(row + 4 * (int64_t)at);
      const any_u32x4_4 a = p[0], b = p[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) o.u[e] = a[e], o.u[4 + e] = b[e];
    } else {
      const any_u32x4_2 a = *(const any_u32x4_2*)(row + 2 * (int64_t)at);
#pragma unroll
      for (int e = 0; e < 4; ++e) o.u[e] = a[e];
    }
    if (by > 0) {
      constexpr int WORDS = K == F32 ? 8 : 4;
#pragma unroll
      for (int s = 4; s >= 1; s /= 2) {
        const int w = K == F32 ? s : s / 2;
#pragma unroll
        for (int e = 0; e < WORDS; ++e) {
          const uint32_t up = e + w < WORDS ? o.u[e + w] : 0u;
          const uint32_t half = e + 1 < WORDS ? o.u[e + 1] : 0u;
          o.u[e] = !(by & s) ? o.u[e] : w ? up : __builtin_amdgcn_alignbit(half, o.u[e], 16);
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int cc = c + e < d ? c + e : 0;
      if constexpr (K == F32) {
        o.u[e] = ((const uint32_t*)row)[cc];
      } else {
        const uint32_t b = ((const uint16_t*)row)[cc];
        o.u[e / 2] = e & 1 ? o.u[e / 2] | b << 16 : b;
      }
    }
  }
}

template <Kind K, bool VEC>
__device__ __forceinline__ void store8(char* row, int c, int d, const Raw<K>& o) {
  if (VEC ? c < d : c + 8 <= d) {
    if constexpr (VEC) {
      uint4* p = (uint4*)(row + (int64_t)c * (K == F32 ? 4 : 2));
      p[0] = make_uint4(o.u[0], o.u[1], o.u[2], o.u[3]);
      if constexpr (K == F32) p[1] = make_uint4(o.u[4], o.u[5], o.u[6], o.u[7]);
    } else if constexpr (K == F32) {
      any_u32x4_4* p = (any_u32x4_4*)(row + 4 * (int64_t)c);
      p[0] = any_u32x4_4{o.u[0], o.u[1], o.u[2], o.u[3]};
      p[1] = any_u32x4_4{o.u[4], o.u[5], o.u[6], o.u[7]};
    } else {
      *(any_u32x4_2*)(row + 2 * (int64_t)c) = any_u32x4_2{o.u[0], o.u[1], o.u[2], o.u[3]};
    }
  } else if constexpr (!VEC) {
    // the row's last one to seven, as four, two and one
    const int n = d - c;
    char* p = row + (int64_t)c * (K == F32 ? 4 : 2);
    uint32_t u0 = o.u[0], u1 = o.u[1];
    if (n <= 0) return;
    if constexpr (K == F32) {
      uint32_t u2 = o.u[2];
      if (n & 4) {
        *(any_u32x4_4*)p = any_u32x4_4{u0, u1, o.u[2], o.u[3]};
        u0 = o.u[4], u1 = o.u[5], u2 = o.u[6], p += 16;
      }
      if (n & 2) {
        *(any_u32x2_4*)p = any_u32x2_4{u0, u1};
        u0 = u2, p += 8;
      }
      if (n & 1) *(uint32_t*)p = u0;
    } else {
      if (n & 4) {
        *(any_u32x2_2*)p = any_u32x2_2{u0, u1};
        u0 = o.u[2], u1 = o.u[3], p += 8;
      }
      if (n & 2) {
        *(any_u32_2*)p = u0;
        u0 = u1, p += 4;
      }
      if (n & 1) *(uint16_t*)p = (uint16_t)u0;
    }
  }
}

// The low bytes of q as elements c .. c + 7.
template <bool VEC>
__device__ __forceinline__ void store8_codes(char* row, int c, int d, const uint32_t q[8]) {
  uint32_t b[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    b[e] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[4 * e + 3], q[4 * e + 2], 0x0c0c0400u),
                                 __builtin_amdgcn_perm(q[4 * e + 1], q[4 * e], 0x0c0c0400u),
                                 0x05040100u);
  if (VEC ? c < d : c + 8 <= d) {
    if constexpr (VEC)
      *(uint2*)(row + c) = make_uint2(b[0], b[1]);
    else
      *(any_u32x2_1*)(row + c) = any_u32x2_1{b[0], b[1]};
  } else if constexpr (!VEC) {
    const int n = d - c;
    char* p = row + c;
    uint32_t u = b[0];
    if (n <= 0) return;
    if (n & 4) *(any_u32_1*)p = u, u = b[1], p += 4;
    if (n & 2) *(any_u16_1*)p = (uint16_t)u, u >>= 16, p += 2;
    if (n & 1) *p = (char)u;
  }
}

template <Kind K>
__device__ __forceinline__ float element(const Raw<K>& o, int e) {
  if constexpr (K == F32)
    return __uint_as_float(o.u[e]);
  else
    return __uint_as_float(e & 1 ? o.u[e / 2] & 0xffff0000u : o.u[e / 2] << 16);
}

// h of eight elements; those past the row's end are 0.
template <Kind X, Kind R, bool VEC>
__device__ __forceinline__ void sum8(const Raw<X>& x, const Raw<R == NONE ? BF16 : R>& r, int c,
                                     int d, float h[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float s = element(x, e);
    if constexpr (R != NONE) s += element(r, e);
    if constexpr (R == BF16) s = __uint_as_float(bf16_bits(s) << 16);
    h[e] = (VEC ? c : c + e) < d ? s : 0.0f;
  }
}

// h as it is stored.
template <Kind R>
__device__ __forceinline__ Raw<R> raw_of(const float h[8]) {
  Raw<R> o;
#pragma unroll
  for (int e = 0; e < (R == F32 ? 8 : 4); ++e)
    o.u[e] = R == F32 ? __float_as_uint(h[e])
                      : __builtin_amdgcn_perm(__float_as_uint(h[2 * e + 1]),
                                              __float_as_uint(h[2 * e]), 0x07060302u);
  return o;
}

// Sum of h^2, maximum of |p|, and 0 p, which is nothing unless p is an infinity
// or a NaN: a maximum passes over NaN, so for the 8-bit scale this joins the
// sum and makes it NaN.  (0 w in float32 would do and is slower: 192 us where
// this takes 182, 16384 x 8192 bf16.)
template <Kind W>
__device__ __forceinline__ void gather8(const float h[8], const Raw<W>& w, double& sum, double& top,
                                        double& odd) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double hd = (double)h[e], p = hd * (double)element(w, e);
    sum = fma(hd, hd, sum);
    top = fmax(top, fabs(p));
    odd = fma(p, 0.0, odd);
  }
}

// What the row's sums give the output.
struct RowOut {
  double rstd, top;
  float c127;
  bool empty, plain;
};

__device__ __forceinline__ RowOut row_out(const NormArgs& a, double sum, double top) {
  RowOut o;
  const double ms = fma(sum, a.inv_d, a.eps);
  o.rstd = ms == 0.0 || ms == INFINITY ? 0.0 : reciprocal_root(ms);
  o.top = top;
  o.c127 = (float)(127.0 * reciprocal(top));
  const float scale = (float)(top * o.rstd * (1.0 / 127.0));
  o.empty = scale == 0.0f;  // also with an ordinary top, where the mean square is large enough
  o.plain = !o.empty && top > 1e-25 && top < 1e30;
  if (a.out_i8 && threadIdx.x == 0) a.scales[blockIdx.x] = o.empty ? 1.0f : scale;
  return o;
}

// A code from float32: adding 1.5 2^23 leaves the nearest whole number (ties to
// even) in a float's low bits.  h w and 127 / P are off by half a step each, so
// their product (formed within a fused addition, not rounded) by less than
// 127 * 2.1 * 2^-24 < 2^-15: unless it is that close to a border, its nearest
// whole number is the code.  Otherwise, and where float32 could overflow or go
// subnormal, the float64 quotient decides.
template <Kind W>
__device__ __forceinline__ void codes8(const RowOut& o, const float h[8], const Raw<W>& w,
                                       uint32_t q[8]) {
  constexpr float MAGIC = 12582912.0f;
  float off = 0.0f;  // farthest from a whole number
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float hw = h[e] * element(w, e), k = fmaf(hw, o.c127, MAGIC);
    off = fmaxf(off, fabsf(fmaf(hw, o.c127, MAGIC - k)));
    q[e] = __float_as_uint(k);
  }
  if (off >= 0.5f - 3.0517578125e-05f || !o.plain) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      q[e] = o.empty ? 0u
                     : (uint32_t)(int)rint(127.0 * ((double)h[e] * (double)element(w, e)) / o.top);
  }
}

template <Kind W>
__device__ __forceinline__ Raw<BF16> bf16_of(const RowOut& o, const float h[8], const Raw<W>& w) {
  Raw<BF16> y;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t b[2];
#pragma unroll
    for (int f = 0; f < 2; ++f)
      b[f] = bf16_bits((float)((double)h[2 * e + f] * (double)element(w, 2 * e + f) * o.rstd));
    y.u[e] = b[0] | b[1] << 16;
  }
  return y;
}

// X, R, W: their types (R NONE: no residual); VPT: elements per thread / 8.
template <Kind X, Kind R, Kind W, int VPT, bool VEC>
__global__ __launch_bounds__((VPT == 4 ? 512 : 1024)) void add_rmsnorm_kernel(NormArgs a) {
  __shared__ double red[2][16];
  constexpr int RB = R == F32 ? 4 : 2;
  const int64_t row = blockIdx.x;
  auto at = [&](int v) __attribute__((always_inline)) {
    return 8 * (v * (int)blockDim.x + (int)threadIdx.x);
  };
  float h[VPT][8];
  Raw<W> w[VPT];
  {
    Raw<X> x[VPT];
    Raw<R == NONE ? BF16 : R> r[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      load8<X, VEC>(a.x + row * a.ldx * (X == F32 ? 4 : 2), at(v), a.d, x[v]);
    if constexpr (R != NONE) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) load8<R, VEC>(a.r + row * a.ldr * RB, at(v), a.d, r[v]);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) load8<W, VEC>(a.w, at(v), a.d, w[v]);
#pragma unroll
    for (int v = 0; v < VPT; ++v) sum8<X, R, VEC>(x[v], r[v], at(v), a.d, h[v]);
  }
  if constexpr (R != NONE) {
    if (a.r_out) {  // R_out may be R: these elements of it have been read
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        store8<R, VEC>(a.r_out + row * a.ldro * RB, at(v), a.d, raw_of<R>(h[v]));
    }
  }
  double sum = 0.0, top = 0.0, odd = 0.0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) gather8<W>(h[v], w[v], sum, top, odd);
  if (a.out_i8) sum += odd;
  fold_row(sum, top, red);
  const RowOut o = row_out(a, sum, top);
  if (!a.out_i8) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      store8<BF16, VEC>(a.out + row * a.ldo * 2, at(v), a.d, bf16_of<W>(o, h[v], w[v]));
    return;
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    uint32_t q[8];
    codes8<W>(o, h[v], w[v], q);
    store8_codes<VEC>(a.out + row * a.ldo, at(v), a.d, q);
  }
}

// Rows longer than REG_D: h is formed twice, from x and r again (R_out, which
// may be R, is written the second time).
template <Kind X, Kind R, Kind W>
__global__ __launch_bounds__(1024) void add_rmsnorm_long_kernel(NormArgs a) {
  __shared__ double red[2][16];
  constexpr int RB = R == F32 ? 4 : 2;
  const int64_t row = blockIdx.x;
  auto load = [&](int c, float h[8], Raw<W>& w) __attribute__((always_inline)) {
    Raw<X> x;
    Raw<R == NONE ? BF16 : R> r;
    load8<X, false>(a.x + row * a.ldx * (X == F32 ? 4 : 2), c, a.d, x);
    if constexpr (R != NONE) load8<R, false>(a.r + row * a.ldr * RB, c, a.d, r);
    load8<W, false>(a.w, c, a.d, w);
    sum8<X, R, false>(x, r, c, a.d, h);
  };
  const int step = 8 * blockDim.x;
  double sum = 0.0, top = 0.0, odd = 0.0;
  for (int c = 8 * threadIdx.x; c < a.d; c += step) {
    float h[8];
    Raw<W> w;
    load(c, h, w);
    gather8<W>(h, w, sum, top, odd);
  }
  if (a.out_i8) sum += odd;
  fold_row(sum, top, red);
  const RowOut o = row_out(a, sum, top);
  for (int c = 8 * threadIdx.x; c < a.d; c += step) {
    float h[8];
    Raw<W> w;
    load(c, h, w);
    if constexpr (R != NONE) {
      if (a.r_out) store8<R, false>(a.r_out + row * a.ldro * RB, c, a.d, raw_of<R>(h));
    }
    if (a.out_i8) {
      uint32_t q[8];
      codes8<W>(o, h, w, q);
      store8_codes<false>(a.out + row * a.ldo, c, a.d, q);
    } else {
      store8<BF16, false>(a.out + row * a.ldo * 2, c, a.d, bf16_of<W>(o, h, w));
    }
  }
}

template <Kind X, Kind R, Kind W, int VPT>
void launch(const NormArgs& a, int64_t m, int threads, bool vec, hipStream_t stream) {
  if (vec)
    hipLaunchKernelGGL((add_rmsnorm_kernel<X, R, W, VPT, true>), dim3((unsigned)m), dim3(threads),
                       0, stream, a);
  else
    hipLaunchKernelGGL((add_rmsnorm_kernel<X, R, W, VPT, false>), dim3((unsigned)m), dim3(threads),
                       0, stream, a);
}

template <Kind X, Kind R, Kind W>
void launch_sized(const NormArgs& a, int64_t m, bool vec, hipStream_t stream) {
  if (a.d > REG_D) {
    hipLaunchKernelGGL((add_rmsnorm_long_kernel<X, R, W>), dim3((unsigned)m), dim3(1024), 0, stream,
                       a);
    return;
  }
  // Enough rows to fill the chip: 256 threads, each with more loads in flight
  // (16384 x 8192 bf16: 181 us with 32 elements per thread, 200 and 249 us with
  // 16 and 8).  Few rows: more threads finish a row sooner, to a point (one row
  // of 8192: 5.4, 4.7 and 5.7 us with 8, 16 and 32; of 16384: 7.5, 7.2, 6.5).
  // (Between, 8193 to 12288, 16 elements are 2 to 8% faster than 32.)
  const int unit = m >= 1024 ? 2048 : 4096;
  const int vpt = a.d <= unit                                         ? 1
                  : a.d <= 2 * unit || (a.d > 8192 && a.d <= 12288) ? 2
                                                                      : 4;
  const int threads = 64 * (int)ceil_div(a.d, 64 * 8 * vpt);
  switch (vpt) {
    case 1: launch<X, R, W, 1>(a, m, threads, vec, stream); break;
    case 2: launch<X, R, W, 2>(a, m, threads, vec, stream); break;
    default: launch<X, R, W, 4>(a, m, threads, vec, stream);
  }
}

template <Kind X, Kind R>
void launch_w(const NormArgs& a, int64_t m, bool w_f32, bool vec, hipStream_t stream) {
  w_f32 ? launch_sized<X, R, F32>(a, m, vec, stream) : launch_sized<X, R, BF16>(a, m, vec, stream);
}

}  // namespace

hipError_t add_rmsnorm_launch(const void* X, int x_dtype, int64_t ldx, const void* R, int r_dtype,
                              int64_t ldr, void* R_out, int64_t ldro, const void* weight,
                              int w_dtype, double eps, int64_t m, int64_t d, void* out,
                              int out_dtype, int64_t ldo, float* out_scales, hipStream_t stream) {
  NormArgs a;
  a.x = (const char*)X, a.r = (const char*)R, a.r_out = (char*)R_out, a.w = (const char*)weight;
  a.out = (char*)out, a.scales = out_scales, a.ldx = ldx, a.ldr = ldr, a.ldro = ldro, a.ldo = ldo;
  a.eps = eps, a.inv_d = 1.0 / (double)d, a.d = (int)d, a.out_i8 = out_dtype == GPTQ_I8;
  const bool xf = x_dtype == GPTQ_F32, rf = r_dtype == GPTQ_F32, wf = w_dtype == GPTQ_F32;
  // 16-byte pieces: every row starts on one, and the row is whole eights
  auto rows16 = [&](const void* p, int64_t ld, int size) {
    return (uintptr_t)p % 16 == 0 && (m == 1 || ld * size % 16 == 0);
  };
  const bool vec = d % 8 == 0 && rows16(X, ldx, xf ? 4 : 2) && (uintptr_t)weight % 16 == 0 &&
                   (!R || rows16(R, ldr, rf ? 4 : 2)) && (!R_out || rows16(R_out, ldro, rf ? 4 : 2)) &&
                   (a.out_i8 ? (uintptr_t)out % 8 == 0 && (m == 1 || ldo % 8 == 0)
                             : rows16(out, ldo, 2));
  // a launch takes less than 2^32 threads: at most 1024 per row, 2^21 rows each
  constexpr int64_t ROWS = (int64_t)1 << 21;
  for (int64_t left = m; left > 0; left -= ROWS) {
    const int64_t n = left < ROWS ? left : ROWS;
    if (!R)
      xf ? launch_w<F32, NONE>(a, n, wf, vec, stream) : launch_w<BF16, NONE>(a, n, wf, vec, stream);
    else if (rf)
      xf ? launch_w<F32, F32>(a, n, wf, vec, stream) : launch_w<BF16, F32>(a, n, wf, vec, stream);
    else
      xf ? launch_w<F32, BF16>(a, n, wf, vec, stream) : launch_w<BF16, BF16>(a, n, wf, vec, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (left > ROWS) {
      a.x += ROWS * ldx * (xf ? 4 : 2);
      if (R) a.r += ROWS * ldr * (rf ? 4 : 2);
      if (R_out) a.r_out += ROWS * ldro * (rf ? 4 : 2);
      a.out += ROWS * ldo * (a.out_i8 ? 1 : 2);
      if (a.out_i8) a.scales += ROWS;
    }
  }
  return hipSuccess;
}

}  // namespace gptq
