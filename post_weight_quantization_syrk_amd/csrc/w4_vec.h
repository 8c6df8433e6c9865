// The products of packed 4-bit weights with a few tokens (m <= 64): bf16 or
// int8 activations, one kernel template for both.
//   Y[i][n] = sx[i] sum_g s[n][g] (sum_{k in g} x q - z[n][g] sum_{k in g} x)
//
// A workgroup owns 16 R weight rows and all tokens.  Its waves take blocks of
// 512 k in turn, each with two buffers of its own in LDS, so that no wave
// waits for another, and their sums meet at the end, in wave order.  (Past 32
// tokens of bf16 those buffers leave room for four to six waves, past 48 for
// three or four, and the tokens, read again for every 16 R rows, are more than
// the weights: in large layers four waves of different rows share them, with a
// barrier per step.  64 tokens through 28672 x 8192: 115 us without, 68 with;
// through 4096 x 11008, 28 and 24.)  A step is 128 k: 64 bytes of each weight row
// and the tokens' pieces, loaded straight into LDS with four neighbouring lanes on
// 64 consecutive bytes.  (Loaded into registers as the matrix instructions want
// them, neighbouring lanes are in different rows, and the vector cache takes one
// lane per cycle: measured 63 accesses per load, 26 us for 16 tokens through 11008
// x 4096.)
// Bound: by no unit alone, but by waits that two waves per SIMD or fewer leave
// open (counters).  16 tokens through 11008 x 4096 take 9.4 us with one scale per
// row, 10.5 in groups of 64 (the weights alone 4.2 at 5.9 TB/s): waves wait for
// loads and barriers 46% of their time (a workgroup's first loads and the waves'
// sums at its end, some 2 us, among it) and for their turn to issue another 19%;
// vector units (codes taken apart, groups' sums scaled) are busy 35% of the time
// over the chip, matrix cores 7%.  37 tokens of int8 through 4099 x 11008 in
// groups of 32: 172 workgroups of seven waves on 256 CUs; waits 37%, vector units
// 37% over the chip, 55% on the CUs that have a workgroup.  32 and 64 tokens of
// bf16 through 28672 x 8192 (50 and 65 us; the weights alone 21): waits 31 and
// 36%, vector units 35 and 34%, matrix cores 16 and 24%.  Three or four
// buffers per wave, four waves with more rows each, and runs of consecutive k per
// wave in place of blocks in turn (8 tokens through 28672 x 8192: 36 us for 33)
// were no faster.
// For int8 X the zero is taken off the codes, four at a time.  For bf16 X that
// would cost an operation per code: x q and x are summed apart (the sum of x by
// the same instruction against ones, shared by all rows), and joined per group.
#pragma once

#include "common.h"

#include <hip/hip_fp16.h>
#include <algorithm>
#include <type_traits>

namespace gptq {
namespace w4vec {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;


struct VecArgs {
  const char* x;        // rows of X
  const float* sx;      // x_scales (int8 X)
  const uint32_t* q;
  const uint16_t* s16;
  const uint16_t* z16;  // null: symmetric
  float* y;
  int64_t ldx;          // bytes
  int m, n, k, ng;
  int vec;              // scales (and zeros) that one aligned load may take: 1, 2, 4 or 8
  int splits, per_split;  // of the row's blocks of 512 k over workgroups
};

// The most that divides a row of scales and its addresses.
inline int scale_vec(const uint16_t* s16, const uint16_t* z16, int ng) {
  const uintptr_t bits = (uintptr_t)s16 | (uintptr_t)z16 | (uintptr_t)(2 * ng);
  return bits % 16 == 0 ? 8 : bits % 8 == 0 ? 4 : bits % 4 == 0 ? 2 : 1;
}

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

// A stored zero as the whole number it is.
__device__ __forceinline__ int whole_zero(uint16_t b) {
  return (int)fminf(fmaxf(rintf(half_bits(b)), -100.0f), 100.0f);
}

// The codes of a word minus their zero, as int8; bits 16..23 of sz hold 128 -
// z.  A byte q + (128 - z) stays within 0..255 for |z| <= 100, so no carry
// crosses bytes; flipping its top bit takes the 128 off again.
__device__ __forceinline__ uint2 code_i8(uint32_t w, uint32_t sz) {
  const uint32_t zc = __builtin_amdgcn_perm(sz, sz, 0x02020202u);
  const uint2 b = code_bytes(w);
  return make_uint2((b.x + zc) ^ 0x80808080u, (b.y + zc) ^ 0x80808080u);
}

constexpr int KCH = 128;   // k per step
constexpr int KBLK = 512;  // k per block: whole scale runs for every group size

// Direct global -> LDS load of 16 bytes per lane: lane l's bytes land at
// lds + 16 l.  In asm, as the compiler would wait for every load in flight
// before any LDS read; the loop waits by count itself.  (M0 may be used for
// LDS one wait state after it is written.)
__device__ __forceinline__ void dma16_at(const void* p, uint32_t lds) {
  const uint32_t lbase = __builtin_amdgcn_readfirstlane(lds);
  __asm__ volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                   :
                   : "v"(p), "s"(lbase)
                   : "memory", "m0");
}

constexpr int LDS_BYTES = 160 * 1024;

// LDS of a wave: two steps' words, and a word with the scale and zero of each
// row and group of a block; and of the waves that share them two steps' tokens.
constexpr int words_bytes(int r, int G) {
  return 2 * 1024 * r + (G == 0 ? 0 : KBLK / G * 16 * r * 4);
}
constexpr int tokens_bytes(bool i8, int nt) { return 2 * 16 * nt * KCH * (i8 ? 1 : 2); }

// LDS of a workgroup of `slots` times rs waves; their sums go where the buffers
// were.
constexpr int group_bytes(bool i8, int nt, int r, int G, int rs, int slots) {
  const int sums = slots * rs * r * nt * 4 * 256;
  const int bytes = slots * (rs * words_bytes(r, G) + tokens_bytes(i8, nt));
  return bytes > sums ? bytes : sums;
}

// Slots that fit: eight waves at most.
constexpr int most_slots(bool i8, int nt, int r, int G, int rs) {
  int slots = 8 / rs;
  while (slots > 1 && group_bytes(i8, nt, r, G, rs, slots) > LDS_BYTES) --slots;
  return slots;
}

template <bool I8, int NT, int R, int G, int RS>
struct Shape {
  static constexpr int XB = I8 ? 1 : 2;
  static constexpr int WBYTES = 1024 * R;             // a step's words
  static constexpr int XBYTES = 16 * NT * KCH * XB;   // a step's tokens
  static constexpr int GPB = G == 0 ? 0 : KBLK / G;   // groups per block
  static constexpr int WORDS = words_bytes(R, G);
  static constexpr int SLOT = RS * WORDS + 2 * XBYTES;
  static constexpr int SLOTS = most_slots(I8, NT, R, G, RS);
  static_assert(group_bytes(I8, NT, R, G, RS, SLOTS) <= LDS_BYTES, "LDS");
};

// I8: int8 X; NT: tiles of 16 tokens; R: tiles of 16 weight rows; G: group
// size, 0 for one group per row; RS: waves that share the tokens' buffers.
template <bool I8, int NT, int R, int G, int RS>
__global__ __launch_bounds__((64 * RS * Shape<I8, NT, R, G, RS>::SLOTS)) void w4_vec_kernel(VecArgs a) {
  typedef typename Types<I8>::acc_t acc_t;
  typedef Shape<I8, NT, R, G, RS> S;
  constexpr bool TR = G == 32 || G == 64;
  constexpr int GPC = G == 0 ? 1 : KCH / G;  // groups per step
  constexpr int XB = S::XB;
  constexpr int XD = (NT * XB * 2 + RS - 1) / RS;  // a wave's direct loads of a step's tokens
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63, w0 = threadIdx.x >> 6;
  const int wave = w0 / RS, waves = (int)(blockDim.x >> 6) / RS, rs = w0 % RS;  // k slot; rows
  const int l16 = lane & 15, h = lane >> 4;
  const int n0 = (blockIdx.x * RS + rs) * 16 * R;
  const int row_bytes = a.k / 2;
  char* const words = smem + wave * S::SLOT + rs * S::WORDS;
  char* const tokens = smem + wave * S::SLOT + RS * S::WORDS;
  const uint32_t words_off = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)words;
  const uint32_t tokens_off = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)tokens;
  uint32_t* const sc = (uint32_t*)(words + 2 * S::WBYTES);

  // steps of this wave: blocks wave, wave + waves, ...; only the row's last
  // block may hold fewer than four
  const int nch = (a.k + KCH - 1) / KCH, b0 = blockIdx.y * a.per_split;
  const int nblk = min((nch + 3) / 4 - b0, a.per_split);
  const int nb = wave < nblk ? (nblk - 1 - wave) / waves + 1 : 0;
  const bool has_last = nb > 0 && 4 * (b0 + wave + waves * (nb - 1)) + 4 > nch;
  const int nst = 4 * nb - (has_last ? 4 - nch % 4 : 0);
  auto chunk = [&](int i) __attribute__((always_inline)) {
    return 4 * (b0 + wave + waves * (i >> 2)) + (i & 3);
  };

  // Direct loads.  Weights: 16 rows of 64 bytes, unit u of row r at u ^ (r / 4
  // mod 4).  Tokens: rows of 128 XB bytes, unit u of token t at u ^ (t mod 16)
  // (bf16) or u ^ (t / 2 mod 8).  Either way 16 lanes that read one unit of 16
  // rows fall on different banks.
  const char* qrow[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    qrow[r] = (const char*)a.q + (int64_t)min(n0 + 16 * r + (lane >> 2), a.n - 1) * row_bytes;
  const int qu = 16 * ((lane & 3) ^ ((lane >> 4) & 3));
  const char* xrow[XD];
  int xu[XD];
#pragma unroll
  for (int i = 0; i < XD; ++i) {
    const int ii = RS * i + rs, t = I8 ? 8 * ii + (lane >> 3) : 4 * ii + (lane >> 4);
    xrow[i] = a.x + (int64_t)min(t, a.m - 1) * a.ldx;
    xu[i] = 16 * (I8 ? (lane & 7) ^ ((t >> 1) & 7) : (lane & 15) ^ (t & 15));
  }
  // loads of tokens that are there
  const int nx = ((I8 ? (a.m + 7) / 8 : (a.m + 3) / 4) + RS - 1 - rs) / RS;
  auto wait_older = [&]() __attribute__((always_inline)) {
    // all but the newest step's R + nx loads (or fewer: that waits longer)
    if (nx == XD)
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(R + XD) : "memory");
    else if (nx >= (XD + 1) / 2)
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(R + (XD + 1) / 2) : "memory");
    else
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(R + 1) : "memory");
  };
  auto issue = [&](int i) __attribute__((always_inline)) {
    const int c = chunk(i);
    const uint32_t dst = words_off + (i & 1) * S::WBYTES;
    const uint32_t xdst = tokens_off + (i & 1) * S::XBYTES + 1024 * rs;
#pragma unroll
    for (int r = 0; r < R; ++r)
      dma16_at(qrow[r] + min(c * (KCH / 2) + qu, row_bytes - 16), dst + 1024 * r);
#pragma unroll
    for (int j = 0; j < XD; ++j) {
      // (whole loads past the last token are left out: their rows hold whatever
      // is there, in sums that are not stored)
      if (j < nx)
        dma16_at(xrow[j] + min(c * KCH * XB + xu[j], a.k * XB - 16), xdst + 1024 * RS * j);
    }
  };
  auto zero_bits = [](uint16_t z) __attribute__((always_inline)) {
    return (uint32_t)(I8 ? 128 - whole_zero(z) : z);
  };
  // The scales and zeros of a block, side by side in LDS, V at a time per lane
  // (a.vec: what their rows' alignment allows); neighbouring lanes take
  // neighbouring pieces of a row.
  auto scales_by = [&](int b, auto vec) __attribute__((always_inline)) {
    constexpr int V = decltype(vec)::value, P = S::GPB / V;  // pieces per row
    constexpr int LD = (16 * R * P + 63) / 64;
    struct alignas(2 * V) Piece {
      uint16_t v[V];
    };
    Piece s[LD], z[LD];
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int e = min(64 * i + lane, 16 * R * P - 1);
      const int64_t o = (int64_t)min(n0 + e / P, a.n - 1) * a.ng + min(b * S::GPB + (e % P) * V, a.ng - V);
      s[i] = *(const Piece*)(a.s16 + o);
      if (a.z16) z[i] = *(const Piece*)(a.z16 + o);
    }
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int e = min(64 * i + lane, 16 * R * P - 1);
#pragma unroll
      for (int v = 0; v < V; ++v)
        sc[((e % P) * V + v) * 16 * R + e / P] =
            s[i].v[v] | zero_bits(a.z16 ? z[i].v[v] : (uint16_t)0x4800) << 16;  // 8
    }
  };
  auto scales = [&](int b) __attribute__((always_inline)) {
    if constexpr (G != 0) {
      if (S::GPB >= 8 && a.vec >= 8)
        scales_by(b, std::integral_constant<int, S::GPB >= 8 ? 8 : 1>());
      else if (a.vec >= 4)
        scales_by(b, std::integral_constant<int, 4>());
      else if (a.vec >= 2)
        scales_by(b, std::integral_constant<int, 2>());
      else
        scales_by(b, std::integral_constant<int, 1>());
    }
  };

  uint32_t row_sz[R];  // G == 0: the row's scale and zero, as in sc
  if constexpr (G == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t n = min(n0 + 16 * r + l16, a.n - 1);
      row_sz[r] = a.s16[n] | zero_bits(a.z16 ? a.z16[n] : (uint16_t)0x4800) << 16;
    }
  }
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
  // tot += s acc, or s (acc - z one) where the zero is still in acc
  auto join = [&](float t, uint32_t sz, auto acc, auto one) __attribute__((always_inline)) {
    const float s = half_bits((uint16_t)sz);
    if constexpr (I8)
      return fmaf(s, (float)acc, t);
    else
      return fmaf(s, fmaf(-half_bits((uint16_t)(sz >> 16)), one, acc), t);
  };

  auto compute = [&](int i) __attribute__((always_inline)) {
    const int c = chunk(i);
    const char* st = words + (i & 1) * S::WBYTES;
    const char* xs = tokens + (i & 1) * S::XBYTES;
    const bool tail = (c + 1) * KCH > a.k;  // pieces past the row's end count as zeros
    uint32_t w[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const char* p = st + 1024 * r + 64 * l16;
      if constexpr (TR) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[r][j] = *(const uint32_t*)(p + 16 * (j ^ ((l16 >> 2) & 3)) + 4 * h);
      } else {
        const uint4 v = *(const uint4*)(p + 16 * (h ^ ((l16 >> 2) & 3)));
        w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
      }
    }
    acc_t one[NT], acc[R][NT];
    auto sz_of = [&](int r, int g) __attribute__((always_inline)) {
      if constexpr (G == 0)
        return row_sz[r];
      else
        return sc[((i & 3) * GPC + g) * 16 * R + 16 * r + l16];
    };
    auto start = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        one[t] = acc_t{0, 0, 0, 0};
        if constexpr (G == 0) one[t] = one0[t];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r][t] = acc_t{0, 0, 0, 0};
          if constexpr (G == 0) acc[r][t] = acc0[r][t];
        }
      }
    };
    auto finish = [&](int g) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t p = sz_of(r, g);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (G == 0) {
            acc0[r][t] = acc[r][t];
            one0[t] = one[t];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              tot[r][t][e] = join(tot[r][t][e], p, acc[r][t][e], one[t][e]);
          }
        }
      }
    };
    if constexpr (!I8) {
      const __bf16 o = (__bf16)1.0f;
      const bf16x8 ones = {o, o, o, o, o, o, o, o};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j % (4 / GPC) == 0) start();
        bf16x8 b[R];
#pragma unroll
        for (int r = 0; r < R; ++r) b[r] = code_bf16(w[r][j]);
        const int u = TR ? 4 * j + h : 4 * h + j;  // 8 k of a token
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint4 v = *(const uint4*)(xs + (16 * t + l16) * 256 + 16 * (u ^ l16));
          if (tail && c * KCH + 8 * u >= a.k) v = make_uint4(0u, 0u, 0u, 0u);
          bf16x8 x;
          __builtin_memcpy(&x, &v, 16);
          one[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, ones, one[t], 0, 0, 0);
#pragma unroll
          for (int r = 0; r < R; ++r)
            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, b[r], acc[r][t], 0, 0, 0);
        }
        if ((j + 1) % (4 / GPC) == 0) finish(j * GPC / 4);
      }
    } else {
      auto two = [](uint2 v) { return (long)(((uint64_t)v.y << 32) | v.x); };
      auto piece = [&](int t, int k) __attribute__((always_inline)) {  // 8 k of a token
        const int u = k >> 4;
        uint2 v = *(const uint2*)(xs + (16 * t + l16) * 128 + 16 * (u ^ ((l16 >> 1) & 7)) + (k & 8));
        if (tail && c * KCH + k >= a.k) v = make_uint2(0u, 0u);
        return v;
      };
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (G == 32) {
#pragma unroll
          for (int jj = 2 * j; jj < 2 * j + 2; ++jj) {
            start();
            long b[R];
#pragma unroll
            for (int r = 0; r < R; ++r) b[r] = two(code_i8(w[r][jj], sz_of(r, jj)));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const long x = two(piece(t, 32 * jj + 8 * h));
#pragma unroll
              for (int r = 0; r < R; ++r)
                acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x32_i8(x, b[r], acc[r][t], 0, 0, 0);
            }
            finish(jj);
          }
        } else {
          if (j % (2 / GPC) == 0) start();
          i32x4 b[R];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t sz = sz_of(r, j * GPC / 2);
            const uint2 p = code_i8(w[r][2 * j], sz), q = code_i8(w[r][2 * j + 1], sz);
            b[r] = i32x4{(int)p.x, (int)p.y, (int)q.x, (int)q.y};
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint2 p = piece(t, TR ? 64 * j + 8 * h : 32 * h + 16 * j);
            const uint2 q = piece(t, TR ? 64 * j + 32 + 8 * h : 32 * h + 16 * j + 8);
            const i32x4 x = {(int)p.x, (int)p.y, (int)q.x, (int)q.y};
#pragma unroll
            for (int r = 0; r < R; ++r)
              acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x, b[r], acc[r][t], 0, 0, 0);
          }
          if ((j + 1) % (2 / GPC) == 0) finish(j * GPC / 2);
        }
      }
    }
  };

  if (nst > 0) issue(0);
  if constexpr (RS == 1) {
    for (int i = 0; i < nst; ++i) {
      // every read of the other buffer has returned before it is written again
      __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if ((i & 3) == 0) scales(chunk(i) >> 2);
      if (i + 1 < nst) {
        issue(i + 1);
        wait_older();
      } else {
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      compute(i);
    }
  } else {
    // slot 0 has the most steps, and every wave comes to each step's barrier
    const int most = 4 * ((nblk - 1) / waves + 1);
    for (int i = 0; i < most; ++i) {
      if ((i & 3) == 0 && i < nst) scales(chunk(i) >> 2);
      // this wave's loads have landed and its reads have returned; behind the
      // barrier that holds for all of them
      __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __syncthreads();
      if (i + 1 < nst) issue(i + 1);
      if (i < nst) compute(i);
    }
  }
  if constexpr (G == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) tot[r][t][e] = join(0.0f, row_sz[r], acc0[r][t][e], one0[t][e]);
  }
  constexpr int PER = R * NT * 4;
  // sums over the buffers: a wave's own, or, where they are shared, all of them
  // once every wave is done
  constexpr int OUT = RS == 1 ? S::SLOT / 4 : PER * 64;  // floats
  static_assert(OUT >= PER * 64, "the wave's sums reuse its buffers");
  if constexpr (RS > 1) __syncthreads();
  float* const out = (float*)smem + (rs * waves + wave) * OUT;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) out[((r * NT + t) * 4 + e) * 64 + lane] = tot[r][t][e];
  __syncthreads();
  for (int e = wave; e < PER; e += waves) {
    float v = 0.0f;
    for (int w = 0; w < waves; ++w) v += ((const float*)smem)[(rs * waves + w) * OUT + e * 64 + lane];
    const int i = e & 3, t = (e >> 2) % NT, r = (e >> 2) / NT;
    const int token = 16 * t + 4 * h + i, n = n0 + 16 * r + l16;
    if (token < a.m && n < a.n) {
      if (I8 && a.splits == 1) v *= a.sx[token];
      a.y[((int64_t)blockIdx.y * a.m + token) * a.n + n] = v;
    }
  }
}

// Y = the splits' products added in split order, times sx where there is one.
// (static: each source that includes this has its own)
static __global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ part,
                                                          const float* __restrict__ sx, int64_t m,
                                                          int n, int splits,
                                                          float* __restrict__ y) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= m * n) return;
  float v = part[e];
  for (int s = 1; s < splits; ++s) v += part[s * m * n + e];
  y[e] = sx ? sx[e / n] * v : v;
}

inline hipError_t join_launch(const float* part, const float* sx, int64_t m, int n, int splits,
                              float* y, hipStream_t stream) {
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)ceil_div(m * n, 256)), dim3(256), 0, stream, part,
                     sx, m, n, splits, y);
  return hipGetLastError();
}

template <bool I8, int NT, int R, int G, int RS>
hipError_t vec_launch_one(const VecArgs& a, hipStream_t stream) {
  typedef Shape<I8, NT, R, G, RS> S;
  const int slots = std::min(S::SLOTS, a.per_split);  // no more than there are blocks
  hipLaunchKernelGGL((w4_vec_kernel<I8, NT, R, G, RS>),
                     dim3((unsigned)ceil_div(a.n, 16 * R * RS), a.splits), dim3(64 * RS * slots),
                     group_bytes(I8, NT, R, G, RS, slots), stream, a);
  return hipGetLastError();
}

template <bool I8, int NT, int R, int RS>
hipError_t vec_launch_g(const VecArgs& a, int G, hipStream_t stream) {
  switch (G) {
    case 32: return vec_launch_one<I8, NT, R, 32, RS>(a, stream);
    case 64: return vec_launch_one<I8, NT, R, 64, RS>(a, stream);
    case 128: return vec_launch_one<I8, NT, R, 128, RS>(a, stream);
    default: return vec_launch_one<I8, NT, R, 0, RS>(a, stream);
  }
}

// Waves share the tokens' buffers only where these are large: bf16, past 32
// tokens (17 to 32: 32 tokens through 28672 x 8192 take 51 us either way).
constexpr int SHARE = 4;
constexpr bool may_share(bool i8, int nt) { return !i8 && nt >= 3; }

struct VecPlan {
  int r;   // tiles of 16 weight rows per wave
  int rs;  // waves that share the tokens' buffers
  int splits, per_split;
  size_t ws_bytes;
};

// Weight rows per workgroup (16 r, or 64 r where waves share the tokens) and
// workgroups that share a row's k, by the least of a time in us.  A step of a
// workgroup's waves takes 0.27 (2 + r) us with 16 tokens and a third more with
// every 16 further ones (4096 x 4096, 16 tokens: 0.8, 1.1 and 1.6 us for r = 1,
// 2, 4); with sharing waves also 6 us to start and end, and more for small
// groups, which are hidden less.  Workgroups beyond what the 256 CUs hold wait
// for a round of their own, which costs 2 us; splits add a launch and their
// sums' bytes.  More rows read X fewer times, fewer of them spread further: 16
// tokens through 11008 x 4096 take 16.1, 13.9, 10.6 and 11.7 us with r = 1 to
// 4, through 4096 x 4096 5.6, 6.7 and 8.9 us with 1, 2 and 4; 64 tokens through
// 1024 x 8192 12.1 us in four splits and 24.5 in one; through 11008 x 4096 23 us
// and 25 with sharing waves, through 8192 x 8192 32 and 29.5, through 16384 x
// 12288 98 and 67.
inline VecPlan vec_plan(bool i8, int64_t m, int64_t n, int64_t k, int G) {
  VecPlan p = {1, 1, 1, 1, 0};
  const int nt = (int)ceil_div(m, 16), nblk = (int)ceil_div(k, KBLK);
  double least = 0.0;
  for (int rs = 1; rs <= SHARE; rs += SHARE - 1)
    for (int r = rs == 1 ? 1 : 2; r <= 4; ++r)
      for (int s = 1; s <= 8 && s <= nblk; ++s) {
        if (rs > 1 && !may_share(i8, nt)) continue;
        const int per = (int)ceil_div(nblk, s), waves = std::min(per, most_slots(i8, nt, r, G, rs));
        const int64_t groups = ceil_div(n, 16 * r * rs) * s;
        const bool several = 2 * group_bytes(i8, nt, r, G, rs, waves) <= LDS_BYTES;  // per CU
        const double rounds =
            several ? std::max(1.0, groups / 256.0) : (double)ceil_div(groups, 256);
        const double steps = 2.0 * (ceil_div(per, waves) + (double)per / waves);  // most and mean
        double us = rounds * 0.27 * (2 + r) * (1.0 + 0.35 * (nt - 1)) * steps;
        if (rs > 1) us = 6.0 + us * (G == 32 ? 1.4 : G == 64 ? 1.25 : 1.0);
        if (!several) us += 2.0 * (rounds - 1.0);  // a round's start and end
        if (s > 1) us += 2.5 + 1e-6 * (double)(m * n) * (s + 1);
        if (least == 0.0 || us < least) {
          least = us;
          p.r = r, p.rs = rs, p.per_split = per, p.splits = (int)ceil_div(nblk, per);
        }
        if (per <= waves) break;  // a wave has one block: no fewer steps
      }
  p.ws_bytes = p.splits > 1 ? (size_t)p.splits * m * n * 4 : 0;
  return p;
}

template <bool I8, int NT>
hipError_t vec_launch_t(const VecArgs& a, int r, int rs, int G, hipStream_t stream) {
  if constexpr (may_share(I8, NT)) {
    if (rs > 1) {
      if (r == 4) return vec_launch_g<I8, NT, 4, SHARE>(a, G, stream);
      if (r == 3) return vec_launch_g<I8, NT, 3, SHARE>(a, G, stream);
      return vec_launch_g<I8, NT, 2, SHARE>(a, G, stream);
    }
  }
  if (r == 4) return vec_launch_g<I8, NT, 4, 1>(a, G, stream);
  if (r == 3) return vec_launch_g<I8, NT, 3, 1>(a, G, stream);
  if (r == 2) return vec_launch_g<I8, NT, 2, 1>(a, G, stream);
  return vec_launch_g<I8, NT, 1, 1>(a, G, stream);
}

template <bool I8>
hipError_t vec_launch(VecArgs a, int G, void* ws, hipStream_t stream) {
  const VecPlan p = vec_plan(I8, a.m, a.n, a.k, G);
  float* const y = a.y;
  if (p.splits > 1) a.y = (float*)ws;
  a.splits = p.splits, a.per_split = p.per_split;
  hipError_t e = a.m <= 16   ? vec_launch_t<I8, 1>(a, p.r, p.rs, G, stream)
                 : a.m <= 32 ? vec_launch_t<I8, 2>(a, p.r, p.rs, G, stream)
                 : a.m <= 48 ? vec_launch_t<I8, 3>(a, p.r, p.rs, G, stream)
                             : vec_launch_t<I8, 4>(a, p.r, p.rs, G, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  return join_launch(a.y, I8 ? a.sx : nullptr, a.m, a.n, p.splits, y, stream);
}

}  // namespace w4vec
}  // namespace gptq
