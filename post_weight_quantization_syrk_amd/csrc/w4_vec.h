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
#include "linear_epi.h"
#include "w4_plan.h"

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
  int vec;              // scales (and zeros) that one aligned load may take: 1, 4 or 8
  int splits, per_split;  // of the row's blocks of 512 k over workgroups
  int slots;              // k slots of a workgroup, at most
};

__host__ __device__ inline Terms terms_of(const VecArgs& a) { return {a.x, a.ldx, a.q, a.s16, a.z16, a.k, a.ng}; }

// How the sums leave: as they are (times sx), or finished by an epilogue.  Gated,
// weight rows u and F + u belong together: a workgroup's row tiles are pairs of
// tiles, first of gate rows, then of the up rows that go with them.
struct Plain {
  static constexpr bool linear = false, gated = false;
};
template <bool GATED>
struct Finished {
  static constexpr bool linear = true, gated = GATED;
  Epilogue e;
};

// Of 8, 4 and 1, the most that divides a row of scales and its addresses.
inline int scale_vec(const uint16_t* s16, const uint16_t* z16, int ng) {
  const uintptr_t bits = (uintptr_t)s16 | (uintptr_t)z16 | (uintptr_t)(2 * ng);
  return bits % 16 == 0 ? 8 : bits % 8 == 0 ? 4 : 1;
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

// The same at a uniform base and a lane's offset.
__device__ __forceinline__ void dma16_from(const void* base, uint32_t voff, uint32_t lds) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const uint32_t blo = __builtin_amdgcn_readfirstlane((uint32_t)b);
  const uint32_t bhi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  const void* sbase = (const void*)(uintptr_t)(((uint64_t)bhi << 32) | blo);
  const uint32_t lbase = __builtin_amdgcn_readfirstlane(lds);
  __asm__ volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                   :
                   : "v"(voff), "s"(sbase), "s"(lbase)
                   : "memory", "m0");
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
template <bool I8, int NT, int R, int G, int RS, class E>
__global__ __launch_bounds__((64 * RS * Shape<I8, NT, R, G, RS>::SLOTS)) void w4_vec_kernel(VecArgs a, E epi) {
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
  // the weight row of this wave's row lr, which may lie past the end; and the
  // nearest that does not
  auto row_at = [&](int lr) __attribute__((always_inline)) {
    if constexpr (E::gated)
      return n0 / 2 + 16 * (lr >> 5) + (lr & 15) + ((lr >> 4) & 1) * epi.e.F;
    else
      return n0 + lr;
  };
  auto valid_row_at = [&](int lr) __attribute__((always_inline)) {
    if constexpr (E::gated)
      return min(n0 / 2 + 16 * (lr >> 5) + (lr & 15), epi.e.F - 1) + ((lr >> 4) & 1) * epi.e.F;
    else
      return min(n0 + lr, a.n - 1);
  };
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
    qrow[r] = (const char*)a.q + (int64_t)valid_row_at(16 * r + (lane >> 2)) * row_bytes;
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
  // The scales and zeros of a block, side by side in LDS, V at a time per lane;
  // neighbouring lanes take neighbouring pieces of a row.  ANY: pieces at any
  // address, that may run into the next row; the matrix's last start earlier instead,
  // and their values go round to their places.
  auto scales_by = [&](int b, auto vec, auto any) __attribute__((always_inline)) {
    constexpr int V = decltype(vec)::value, P = S::GPB / V;  // pieces per row
    constexpr bool ANY = decltype(any)::value;
    constexpr int LD = (16 * R * P + 63) / 64;
    struct alignas(ANY ? 2 : 2 * V) Piece {
      uint16_t v[V];
    };
    Piece s[LD], z[LD];
    int early[LD];
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int e = min(64 * i + lane, 16 * R * P - 1), j = b * S::GPB + (e % P) * V;
      int64_t o = (int64_t)valid_row_at(e / P) * a.ng + min(j, a.ng - (ANY ? 1 : V));
      early[i] = 0;
      if constexpr (ANY) {
        early[i] = (int)max(o + V - (int64_t)a.n * a.ng, (int64_t)0);
        o -= early[i];
      }
      s[i] = *(const Piece*)(a.s16 + o);
      if (a.z16) z[i] = *(const Piece*)(a.z16 + o);
    }
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int e = min(64 * i + lane, 16 * R * P - 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int at = (e % P) * V + (ANY ? (v - early[i]) & (V - 1) : v);
        const uint32_t both = s[i].v[v] | zero_bits(a.z16 ? z[i].v[v] : (uint16_t)0x4800) << 16;  // 8
        sc[at * 16 * R + e / P] = ANY && b * S::GPB + at >= a.ng ? 0 : both;  // (another row's)
      }
    }
  };
  // Aligned where the rows are; else, for bf16 tokens, at any address with groups of 32
  // (31 tokens through 25020 x 5216, gated, 58 us, with 2 bytes a load 85; 16 through 8192
  // x 11040 20.8 and 26.5) or many weight rows (15 tokens, groups of 64: 9700 x 5440 16%
  // less than 2 bytes a load, 5500 x 5440 4%, 4100 x 2752 7% more; of 128: 9700 x 5504 10%
  // less, 4100 x 2432 2% more).  One by one otherwise, and for int8 tokens (15 tokens, groups
  // of 64, 11436 x 5440: 11.1 us, at any address 11.8; 2684 x 5440 7.4 and 8.3).
  auto scales = [&](int b) __attribute__((always_inline)) {
    constexpr std::false_type aligned{};
    if constexpr (G != 0) {
      if (S::GPB >= 8 && a.vec >= 8) {
        scales_by(b, std::integral_constant<int, S::GPB >= 8 ? 8 : 1>(), aligned);
      } else if (a.vec >= 4) {
        scales_by(b, std::integral_constant<int, 4>(), aligned);
      } else {
        if constexpr (!I8) {
          if ((G == 32 || a.n >= 5000) && (int64_t)a.n * a.ng >= 8)
            return scales_by(b, std::integral_constant<int, S::GPB >= 8 ? 8 : 4>(), std::true_type());
        }
        scales_by(b, std::integral_constant<int, 1>(), aligned);
      }
    }
  };

  uint32_t row_sz[R];  // G == 0: the row's scale and zero, as in sc
  if constexpr (G == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t n = valid_row_at(16 * r + l16);
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
  auto summed = [&](int e) __attribute__((always_inline)) {
    float v = 0.0f;
    for (int w = 0; w < waves; ++w) v += ((const float*)smem)[(rs * waves + w) * OUT + e * 64 + lane];
    return v;
  };
  // Finished outputs: a first round over those whose sums are finite; a second, where
  // any was not, over those.  (A check with a branch for each sum took 3 us of 30 of 48
  // tokens through 28672 x 4096.)
  auto finished = [&](auto second) __attribute__((always_inline)) {
    constexpr bool SECOND = decltype(second)::value;
    bool odd = false;
    if constexpr (E::gated) {
      for (int q = wave; q < PER / 2; q += waves) {
        const int i = q & 3, t = (q >> 2) % NT, r = (q >> 2) / NT * 2;
        const int token = 16 * t + 4 * h + i, u = row_at(16 * r + l16);
        float v0 = summed((r * NT + t) * 4 + i), v1 = summed(((r + 1) * NT + t) * 4 + i);
        bool now = token < a.m && u < epi.e.F, fin = is_finite(v0) && is_finite(v1);
        odd = odd || (now && !fin);
        now = now && fin != SECOND;
        if constexpr (SECOND) {
          right_odd_sums(terms_of(a), now, token, u, v0);
          right_odd_sums(terms_of(a), now, token, epi.e.F + u, v1);
        }
        if (now) finish<true>(epi.e, token, u, v0, v1);
      }
    } else if constexpr (E::linear) {
      for (int e = wave; e < PER; e += waves) {
        float v = summed(e);
        const int i = e & 3, t = (e >> 2) % NT, r = (e >> 2) / NT;
        const int token = 16 * t + 4 * h + i, n = row_at(16 * r + l16);
        bool now = token < a.m && n < a.n, fin = is_finite(v);
        odd = odd || (now && !fin);
        now = now && fin != SECOND;
        if constexpr (SECOND) right_odd_sums(terms_of(a), now, token, n, v);
        if (now) finish<false>(epi.e, token, n, v, 0.0f);
      }
    }
    return __any(odd);
  };
  if constexpr (E::linear) {
    if (a.splits == 1) {
      if (__builtin_expect(finished(std::false_type()), 0)) finished(std::true_type());
      return;
    }
  }
  for (int e = wave; e < PER; e += waves) {
    float v = summed(e);
    const int i = e & 3, t = (e >> 2) % NT, r = (e >> 2) / NT;
    const int token = 16 * t + 4 * h + i, n = row_at(16 * r + l16);
    bool in = token < a.m && n < a.n;
    if constexpr (E::gated) in = in && n - (r & 1) * epi.e.F < epi.e.F;
    if (in) {
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

template <bool I8, int NT, int R, int G, int RS, class E>
hipError_t vec_launch_one(const VecArgs& a, const E& e, hipStream_t stream) {
  typedef Shape<I8, NT, R, G, RS> S;
  // no more waves than there are blocks
  const int slots = std::min(std::min(S::SLOTS, a.per_split), a.slots);
  hipLaunchKernelGGL((w4_vec_kernel<I8, NT, R, G, RS, E>),
                     dim3((unsigned)ceil_div(a.n, 16 * R * RS), a.splits), dim3(64 * RS * slots),
                     group_bytes(I8, NT, R, G, RS, slots), stream, a, e);
  return hipGetLastError();
}

template <bool I8, int NT, int R, int RS, class E>
hipError_t vec_launch_g(const VecArgs& a, int G, const E& e, hipStream_t stream) {
  switch (G) {
    case 32: return vec_launch_one<I8, NT, R, 32, RS>(a, e, stream);
    case 64: return vec_launch_one<I8, NT, R, 64, RS>(a, e, stream);
    case 128: return vec_launch_one<I8, NT, R, 128, RS>(a, e, stream);
    default: return vec_launch_one<I8, NT, R, 0, RS>(a, e, stream);
  }
}

template <bool I8, int NT, class E>
hipError_t vec_launch_t(const VecArgs& a, int r, int rs, int G, const E& e, hipStream_t stream) {
  if constexpr (may_share(I8, NT)) {
    if (rs > 1) {
      if (r == 4) return vec_launch_g<I8, NT, 4, SHARE>(a, G, e, stream);
      if constexpr (!E::gated) {
        if (r == 3) return vec_launch_g<I8, NT, 3, SHARE>(a, G, e, stream);
      }
      return vec_launch_g<I8, NT, 2, SHARE>(a, G, e, stream);
    }
  }
  if (r == 4) return vec_launch_g<I8, NT, 4, 1>(a, G, e, stream);
  if constexpr (!E::gated) {
    if (r == 3) return vec_launch_g<I8, NT, 3, 1>(a, G, e, stream);
    if (r == 1) return vec_launch_g<I8, NT, 1, 1>(a, G, e, stream);
  }
  return vec_launch_g<I8, NT, 2, 1>(a, G, e, stream);
}

// The product; with splits their sums are left in ws, for the caller to join.
template <bool I8, class E>
hipError_t vec_launch_parts(VecArgs a, const VecPlan& p, int G, void* ws, const E& e,
                            hipStream_t stream) {
  if (p.splits > 1) a.y = (float*)ws;
  a.splits = p.splits, a.per_split = p.per_split, a.slots = p.slots;
  return a.m <= 16   ? vec_launch_t<I8, 1>(a, p.r, p.rs, G, e, stream)
         : a.m <= 32 ? vec_launch_t<I8, 2>(a, p.r, p.rs, G, e, stream)
         : a.m <= 48 ? vec_launch_t<I8, 3>(a, p.r, p.rs, G, e, stream)
                     : vec_launch_t<I8, 4>(a, p.r, p.rs, G, e, stream);
}

template <bool I8>
hipError_t vec_launch(const VecArgs& a, int G, void* ws, hipStream_t stream) {
  const VecPlan p = vec_plan(I8, a.m, a.n, a.k, G);
  const hipError_t e = vec_launch_parts<I8>(a, p, G, ws, Plain{}, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  return join_launch((const float*)ws, I8 ? a.sx : nullptr, a.m, a.n, p.splits, a.y, stream);
}

// The same with an epilogue.
template <bool I8, bool GATED>
hipError_t vec_finish_launch(const VecArgs& a, int G, void* ws, const Epilogue& epi,
                             hipStream_t stream) {
  const VecPlan p = vec_plan(I8, a.m, a.n, a.k, G, true, GATED);
  const hipError_t e = vec_launch_parts<I8>(a, p, G, ws, Finished<GATED>{epi}, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  return join_finish_launch<GATED>((const float*)ws, a.m, a.n, p.splits, epi, terms_of(a), stream);
}

}  // namespace w4vec
}  // namespace gptq
