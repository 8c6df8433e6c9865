// The W4A16 product with its epilogue, for more than a few tokens:
//   Y = act(X W_hat^T + bias) + residual, or gated by pairs of weight rows
//   (linear_epi.h), W_hat[n][k] = s[n][k/g] (q[n][k] - z[n][k/g]).
//
// q - z is exact in bf16, so products with X are exact in float32; a group's sum
// stands by itself and is scaled into the total with one operation per sum
// (v_mfma_f32_32x32x16_bf16: for every product of 32 x 32 x 16 as many vector
// operations as a group has sixteens of k go into 16, so 8 at groups of 32, 4 at 64, 2
// at 128; four cost nothing beside a product, eight take as long as it).
//
// Two forms of the weights.  Four bits: each wave takes its own 32 weight rows apart,
// once, for up to 256 rows of X; chunks of 64 k of X and of the words come to LDS by
// direct loads, up to three ahead.  Eight bits first (`Wide`) for many rows: a wave has
// 64 weight rows, and two codes become bf16 with one operation.
//
// 8192 tokens through 57344 x 8192, groups of 128, gated, SiLU: 6.8 to 7.3 ms by card, 1.06 to 1.13 PF/s, of
// which 0.15 ms make the weights wide; a library bf16 product of 8192^3 reaches 1.29.
// The clock falls to some 1.65 GHz there (power), at which the matrix cores are busy
// 61% of the cycles.  515 tokens through 4099 x 11008, groups of 32: 91 to 99 us by
// card, of which the join of five splits takes 11: 14 vector operations to a product
// (eight scale its sums, the rest are the codes' and addresses) are busy 45% of the
// cycles, the matrix cores 25%, and waves wait 24% of theirs, at a workgroup's start
// and end above all.  96 tokens through 4096 x
// 4096: 24 us, of which launches, a workgroup's start and end take two thirds.
#include "common.h"
#include "kernels.h"
#include "linear_plan.h"
#include "w4_dot.h"

namespace gptq {

using namespace linear;

namespace {

// Columns of a tile in the order in which it takes weight rows: gated, 32 gate
// rows, then the 32 up rows that go with them.
template <bool GATED>
__device__ __forceinline__ int64_t weight_row(int64_t c, int F) {
  return GATED ? (c >> 6) * 32 + (c & 31) + ((c >> 5) & 1) * F : c;
}
template <bool GATED>
__device__ __forceinline__ bool weight_row_in(int64_t c, int F) {
  return GATED ? (c >> 6) * 32 + (c & 31) < F : c < F;
}

template <bool GATED>
__global__ __launch_bounds__(256) void widen_kernel(Wide w, int F, int K, int G,
                                                    const uint32_t* __restrict__ Q,
                                                    const uint16_t* __restrict__ S16,
                                                    const uint16_t* __restrict__ Z16,
                                                    char* __restrict__ ws) {
  const int64_t pieces = w.cols * w.nch * 2;  // of 32 k
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t < pieces) {
    const int64_t c = t / (2 * w.nch);
    const int piece = (int)(t - c * (2 * w.nch)), k = 32 * piece;
    const int r = (int)(c & 31);
    uint4 o[2] = {};
    if (k < K && weight_row_in<GATED>(c, F)) {
      const int64_t row = weight_row<GATED>(c, F);
      const uint4 v = *(const uint4*)((const char*)Q + row * (K / 2) + k / 2);
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      const float z = Z16 ? w4vec::half_bits(Z16[row * w.ng + k / G]) : 8.0f;
      uint32_t out[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = (float)((in[i / 2] >> (16 * (i & 1) + 4 * j)) & 15u) - z;
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
        out[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], b, true);
      }
      o[0] = make_uint4(out[0], out[1], out[2], out[3]);
      o[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
    char* const panel = ws + ((c >> 5) * w.nch + (piece >> 1)) * 2048 + r * 64;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *(uint4*)(panel + 16 * ((2 * (piece & 1) + j) ^ ((r >> 2) & 3))) = o[j];
  } else if (t - pieces < w.cols * w.ng) {
    const int64_t i = t - pieces;
    const int g = (int)(i / w.cols);
    const int64_t c = i - g * w.cols;
    ((float*)(ws + w.scales))[i] =
        weight_row_in<GATED>(c, F) ? w4vec::half_bits(S16[weight_row<GATED>(c, F) * w.ng + g]) : 0.0f;
  }
}

// The eight codes of a word minus the zero, as bf16 in k order: even and odd
// codes come apart by masks, each byte converts by itself (the empty asm keeps
// the masks from becoming per-code bit-field extracts), and the upper halves of
// two differences, exact, are joined by a byte permute.
__device__ __forceinline__ bf16x8 minus_zero(uint32_t w, float z) {
  uint32_t ev = w & 0x0f0f0f0fu, od = (w >> 4) & 0x0f0f0f0fu;
  asm("" : "+v"(ev), "+v"(od));
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = (float)((ev >> (8 * j)) & 0xffu) - z;
    const float hi = (float)((od >> (8 * j)) & 0xffu) - z;
    o[j] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
  }
  bf16x8 r;
  __builtin_memcpy(&r, o, sizeof(r));
  return r;
}

// Eight of the wide weights.
__device__ __forceinline__ bf16x8 from_wide(uint32_t a, uint32_t b) {
  const w4vec::bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const w4vec::bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const w4vec::bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const w4vec::bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

struct Args {
  const char* x;
  int64_t ldx;    // bytes
  const uint32_t* q;
  const uint16_t *s16, *z16;  // z16 null: symmetric
  const char* wide;           // the weights in eight bits, or null
  const float* scales;        // and their scales [ng][cols]
  int64_t cols;
  float* part;    // splits' sums [splits][M][N], null: finished here
  Epilogue e;
  int64_t M;
  int N, K, ng;
  int tiles_m, tiles_n;
  int splits, per_split;  // of the chunks
};

constexpr int BLOCK = 8;  // groups whose scales a wave has in LDS
constexpr int SCALES = 4 * BLOCK * 32 * 4;
constexpr int LDS_BYTES = 80 * 1024;  // two workgroups on a CU

template <int MI, bool WIDE>
struct Shape {
  static constexpr int ABYTES = 32 * MI * 2 * KCH, BBYTES = tile_n(WIDE) * KCH / (WIDE ? 1 : 2);
  static constexpr int STAGE = ABYTES + BBYTES;
  static constexpr int LOADS = MI + 1;  // of a wave per chunk (4-bit weights)
  // chunks in LDS: two of the wide weights (their scales come by ordinary loads,
  // which the compiler waits for by waiting for all), else as many as fit, up to four
  static constexpr int FIT = (LDS_BYTES - SCALES) / STAGE;
  static constexpr int BUFS = WIDE ? 2 : FIT < 4 ? FIT : 4;
  static_assert(BUFS >= 2 && BUFS * STAGE <= LDS_BYTES, "two buffers");
};

// A barrier for LDS alone: __syncthreads() also waits for the stores that are out,
// 1 us for every 32 rows that leave.
__device__ __forceinline__ void lds_barrier() {
  __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ const uint4 zeros = {};  // a unit of X past the rows' end

// Four waves side by side, each all 32 MI rows of X by 32 weight rows: a wave
// takes the codes of its own weight rows apart, and none twice.  G: group size,
// 0 for one group per row.
template <int MI, int G, bool GATED, bool WIDE>
__device__ __forceinline__ void tile_product(const Args& a, char* lds, int64_t m0, int64_t c0,
                                             int split) {
  typedef Shape<MI, WIDE> S;
  constexpr int GPC = G == 32 ? 2 : 1;  // groups in a chunk
  constexpr int STAGE = S::STAGE, BUFS = S::BUFS, ABYTES = S::ABYTES;
  constexpr int NI = blocks_n(WIDE), TN = tile_n(WIDE), BL = MI * NI;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, l32 = lane & 31;
  const int nch = (a.K + KCH - 1) / KCH, ch0 = split * a.per_split,
            ch1 = min(nch, ch0 + a.per_split);
  const int64_t wcol = c0 + 32 * NI * wave;  // this wave's first column
  const int F = a.e.F;

  // direct loads, 1 KB each: 8 rows of X, or 32 weight rows, at units that put
  // 16 rows on different banks; bases are uniform, lanes have 32-bit offsets
  const char* xbase = a.x + m0 * a.ldx;
  auto xu = [&](int j) __attribute__((always_inline)) {  // of row 8 (MI wave + j) + lane / 8
    return 16 * ((lane & 7) ^ ((4 * (MI * wave + j) + (lane >> 4)) & 7));
  };
  uint32_t xoff[MI];
#pragma unroll
  for (int j = 0; j < MI; ++j) {
    const int r = 8 * (MI * wave + j) + (lane >> 3);
    xoff[j] = (uint32_t)min((int64_t)r, a.M - 1 - m0) * (uint32_t)a.ldx + xu(j);
  }
  // columns past the last: copies of the last valid row of this wave, or of row 0
  const int64_t row0 = weight_row<GATED>(wcol, F);
  const int there = weight_row_in<GATED>(wcol, F)
                        ? (int)min((int64_t)32, F - (GATED ? (wcol >> 6) * 32 : wcol)) : 0;
  const char* qbase = (const char*)a.q + (there ? row0 : 0) * (a.K / 2);
  const uint32_t qrow = (uint32_t)min(lane >> 1, max(there - 1, 0)) * (uint32_t)(a.K / 2);
  const int qu = 16 * ((lane & 1) ^ ((lane >> 4) & 1));
  const char* const wbase = a.wide + (wcol >> 5) * nch * 2048;
  auto issue = [&](int c, int buf) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + buf * STAGE;
    const char* const xb = xbase + (int64_t)c * (2 * KCH);
    const char* const qb = qbase + (int64_t)c * (KCH / 2);
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < 2 * NI; ++j)
        w4vec::dma16_from(wbase + ((int64_t)(j >> 1) * nch + c) * 2048 + 1024 * (j & 1), lane * 16,
                          dst + ABYTES + (2 * NI * wave + j) * 1024);
    }
    if ((c + 1) * KCH <= a.K) {
#pragma unroll
      for (int j = 0; j < MI; ++j) w4vec::dma16_from(xb, xoff[j], dst + (MI * wave + j) * 1024);
      if constexpr (!WIDE) w4vec::dma16_from(qb, qrow + qu, dst + ABYTES + wave * 1024);
    } else {
      // a last chunk that is not whole: past the rows' end X is zeros (a copy might be
      // infinite, and a weight of 0 times that is a NaN), words are copies
      const int xmost = 2 * a.K - 16 - c * 2 * KCH, qmost = a.K / 2 - 16 - c * (KCH / 2);
#pragma unroll
      for (int j = 0; j < MI; ++j) {
        const char* const from = xb + xoff[j];
        w4vec::dma16_at(xu(j) <= xmost ? from : (const char*)&zeros, dst + (MI * wave + j) * 1024);
      }
      if constexpr (!WIDE) w4vec::dma16_from(qb, qrow + min(qu, qmost), dst + ABYTES + wave * 1024);
    }
  };
  // The scales and zeros of BLOCK groups of the wave's rows, a word each in LDS:
  // lane half 0 loads a row's scales, half 1 its zeros, one block ahead.
  constexpr int CPB = G == 0 ? 1 : BLOCK * G / KCH;  // chunks per block
  uint32_t* const sc = (uint32_t*)(lds + BUFS * STAGE) + wave * BLOCK * 32;
  const int64_t mrow = there ? row0 + min(l32, there - 1) : 0;
  const uint16_t* const meta = (h && a.z16 ? a.z16 : a.s16) + mrow * a.ng;
  const bool eights = a.z16 == nullptr && h;  // symmetric: zeros are 8
  uint32_t ahead[4];
  auto fetch = [&](int b) __attribute__((always_inline)) {
    if (a.ng >= BLOCK) {
      // the row's last block starts earlier instead of running past its end
      __builtin_memcpy(ahead, meta + min(b * BLOCK, a.ng - BLOCK), 16);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ahead[j] = meta[min(2 * j, a.ng - 1)] | (uint32_t)meta[min(2 * j + 1, a.ng - 1)] << 16;
    }
    if (eights) ahead[0] = ahead[1] = ahead[2] = ahead[3] = 0x48004800u;
  };
  auto first_group = [&](int b) __attribute__((always_inline)) {
    return a.ng >= BLOCK ? min(b * BLOCK, a.ng - BLOCK) : 0;
  };
  auto publish = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // scales of groups 2j, 2j + 1 in every lane, and zeros
      const w4vec::u32x2 r = __builtin_amdgcn_permlane32_swap(ahead[j], ahead[j], false, false);
      if (h == (j >> 1)) {
        sc[2 * j * 32 + l32] = __builtin_amdgcn_perm(r[1], r[0], 0x05040100u);
        sc[(2 * j + 1) * 32 + l32] = __builtin_amdgcn_perm(r[1], r[0], 0x07060302u);
      }
    }
  };
  uint32_t row_sz = 0;
  float next[NI * GPC];  // wide: the scales of the chunk to come (of the row, G = 0)
  const float* const wscale = a.scales + wcol + l32;
  auto fetch_wide = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NI * GPC; ++i)
      next[i] = wscale[(G == 0 ? 0 : min(c * KCH / (G ? G : 1) + i % GPC, a.ng - 1)) * a.cols + 32 * (i / GPC)];
  };
  if constexpr (WIDE) {
    fetch_wide(ch0);
  } else if constexpr (G == 0) {
    row_sz = a.s16[mrow] | (uint32_t)(a.z16 ? a.z16[mrow] : 0x4800) << 16;
  } else {
    fetch(ch0 / CPB);
  }

  f32x16 tot[BL];  // blocks, ni the faster index
#pragma unroll
  for (int b = 0; b < BL; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) tot[b][i] = 0.0f;
#pragma unroll
  for (int i = 0; i < BUFS - 1; ++i)
    if (ch0 + i < ch1) issue(ch0 + i, i);
  int buf = 0, fill = BUFS - 1;
  for (int c = ch0; c < ch1; ++c) {
    // chunk c has landed, and chunk c - 1's buffer is read
    if (c + BUFS - 2 < ch1)
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"((BUFS - 2) * S::LOADS) : "memory");
    else
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    float scale[NI * GPC], z[GPC];
    if constexpr (WIDE && G != 0) {
      // (here, so that the compiler waits for them before more loads are out)
#pragma unroll
      for (int g = 0; g < NI * GPC; ++g) {
        scale[g] = next[g];
        asm volatile("" : "+v"(scale[g]));
      }
    }
    __syncthreads();
    if (c + BUFS - 1 < ch1) issue(c + BUFS - 1, fill);
    if constexpr (WIDE && G != 0) {
      if (c + 1 < ch1) fetch_wide(c + 1);
    }
    fill = fill + 1 == BUFS ? 0 : fill + 1;
    const char* la = lds + buf * STAGE + l32 * 2 * KCH;
    const char* lb = lds + buf * STAGE + ABYTES + (32 * NI * wave + l32) * (WIDE ? KCH : KCH / 2);
    int sc_at[GPC] = {};  // of the chunk's groups; past the row's end, of its last
    if constexpr (G != 0 && !WIDE) {
      const int b = c / CPB;
      if (c == ch0 || c % CPB == 0) {
        publish();
        if ((b + 1) * CPB < ch1) fetch(b + 1);
      }
#pragma unroll
      for (int g = 0; g < GPC; ++g)
        sc_at[g] = (min(c * KCH / G + g, a.ng - 1) - first_group(b)) * 32 + l32;
    }
    buf = buf + 1 == BUFS ? 0 : buf + 1;
    const int sw = (l32 >> 3) & 1;
    // MFMA q of a chunk takes, in lane half h, unit u of X: with groups of 32
    // the two halves share 32 consecutive k, otherwise 64
    auto unit = [&](int q) __attribute__((always_inline)) {
      return G == 32 ? 4 * (q >> 1) + 2 * h + (q & 1) : 4 * h + q;
    };
    auto xfrag = [&](int mi, int q) __attribute__((always_inline)) {
      return *(const bf16x8*)(la + mi * 32 * 2 * KCH + 16 * (unit(q) ^ ((l32 >> 1) & 7)));
    };
    const bool tail = (c + 1) * KCH > a.K;  // past the row's end: zeros
    bf16x8 bf[NI * 4];
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < 2 * NI; ++i) {
        const int j = i & 1, u = G == 32 ? 2 * j + h : 2 * h + j;
        const uint4 v = *(const uint4*)(lb + (i >> 1) * 32 * KCH + 16 * (u ^ ((l32 >> 2) & 3)));
        bf[2 * i] = from_wide(v.x, v.y);
        bf[2 * i + 1] = from_wide(v.z, v.w);
      }
    } else {
#pragma unroll
      for (int g = 0; g < GPC; ++g) {
        const uint32_t v = G == 0 ? row_sz : sc[sc_at[g]];
        scale[g] = w4vec::half_bits((uint16_t)v);
        z[g] = w4vec::half_bits((uint16_t)(v >> 16));
        asm("" : "+v"(scale[g]), "+v"(z[g]));  // or every product converts it again
      }
      uint32_t w[4];
      if constexpr (G == 32) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint2 v = *(const uint2*)(lb + 16 * (j ^ sw) + 8 * h);
          w[2 * j] = v.x, w[2 * j + 1] = v.y;
        }
      } else {
        const uint4 v = *(const uint4*)(lb + 16 * (h ^ sw));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) bf[q] = minus_zero(w[q], z[G == 32 ? q >> 1 : 0]);
      if (tail) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c * KCH + 8 * unit(q) >= a.K) bf[q] = bf16x8{};
      }
    }
    if constexpr (G == 0) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8 x = xfrag(mi, q);
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            tot[mi * NI + ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, bf[4 * ni + q],
                                                                        tot[mi * NI + ni], 0, 0, 0);
        }
    } else {
      // step s multiplies for one block and one group while the step before it is
      // scaled into its total, behind half of the step's products: the sum has
      // left the matrix cores by then
      constexpr int PER = NI * GPC, STEPS = MI * PER, QPS = 4 / GPC;
      bf16x8 af[2][4];
      f32x16 acc[2];
#pragma unroll
      for (int q = 0; q < 4; ++q) af[0][q] = xfrag(0, q);
#pragma unroll
      for (int s = 0; s <= STEPS; ++s) {
        const int mi = s / PER, ni = s % PER / GPC, g = s % GPC;
        __builtin_amdgcn_sched_barrier(0);
        if (s < STEPS) {
          // its share of the next 32 rows' units
          if (mi + 1 < MI) {
#pragma unroll
            for (int q = s % PER * 4 / PER; q < (s % PER + 1) * 4 / PER; ++q)
              af[(mi + 1) & 1][q] = xfrag(mi + 1, q);
          }
          acc[s & 1] = f32x16{};
#pragma unroll
          for (int q = 0; q < QPS; ++q)
            acc[s & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                af[mi & 1][g * QPS + q], bf[4 * ni + g * QPS + q], acc[s & 1], 0, 0, 0);
        }
        if (s > 0) {
          const int p = s - 1;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            tot[p / GPC][i] = fmaf(scale[p % PER], acc[p & 1][i], tot[p / GPC][i]);
        }
#pragma unroll
        for (int q = 0; q < QPS; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);        // an LDS read
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);        // a product
          if (2 * q >= QPS)
            __builtin_amdgcn_sched_group_barrier(0x002, 32 / QPS, 0); // its share of the scaling
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (G == 0) {
#pragma unroll
    for (int b = 0; b < BL; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        tot[b][i] *= WIDE ? next[b % NI] : w4vec::half_bits((uint16_t)row_sz);
  }
  // Out by way of LDS, 32 rows at a time, four columns to a thread: whole rows of
  // Y are stored, and the epilogue's code is there once.
  constexpr int OUT = GATED ? TN / 2 : TN;  // columns of Y
  constexpr int TPR = OUT / 4;              // threads per row
  const int64_t u0 = GATED ? c0 / 2 : c0;
  float* const sums = (float*)lds;
  const int col = 4 * (threadIdx.x % TPR);
  const int lcol = GATED ? 64 * (col >> 5) + (col & 31) : col;
  const int ncol = (int)min((int64_t)4, F - (u0 + col));  // of these columns, those that are there
  __syncthreads();
#pragma unroll 1
  for (int mi = 0; mi < MI; ++mi) {
#pragma unroll
    for (int j = 0; j < MI; ++j) {
      if (j != mi) continue;
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sums[(8 * (i >> 2) + 4 * h + (i & 3)) * TN + 32 * (NI * wave + ni) + l32] =
              tot[j * NI + ni][i];
    }
    lds_barrier();
    if (a.part) {
      // columns a thread apart, so that stores are of neighbours whatever N's alignment
#pragma unroll
      for (int r = 0; r < 32; r += 256 / TPR) {
        const int rt = r + (int)threadIdx.x / TPR;
        const int64_t row = m0 + 32 * mi + rt;
        float* const o = a.part + ((int64_t)split * a.M + row) * a.N + u0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = (int)(threadIdx.x % TPR) + TPR * i, l = GATED ? 64 * (k >> 5) + (k & 31) : k;
          if (row >= a.M || k >= F - u0) continue;
          o[k] = sums[rt * TN + l];
          if constexpr (GATED) o[F + k] = sums[rt * TN + l + 32];
        }
      }
      lds_barrier();
      continue;
    }
#pragma unroll 1
    for (int r = threadIdx.x / TPR; r < 32; r += 256 / TPR) {
      const int64_t row = m0 + 32 * mi + r;
      if (row >= a.M || ncol <= 0) break;
      const float4 p = *(const float4*)(sums + r * TN + lcol);
      float v0[4] = {p.x, p.y, p.z, p.w}, v1[4] = {};
      if constexpr (GATED) {
        const float4 q = *(const float4*)(sums + r * TN + lcol + 32);
        v1[0] = q.x, v1[1] = q.y, v1[2] = q.z, v1[3] = q.w;
      }
      finish4<GATED>(a.e, row, u0 + col, ncol, v0, v1);
    }
    lds_barrier();
  }
}

template <int G, bool GATED, bool WIDE>
__global__ __launch_bounds__(256, 2) void linear_kernel(Args a) {
  __shared__ __attribute__((aligned(1024))) char lds[LDS_BYTES];
  // consecutive workgroups go to the eight XCDs in turn: each XCD takes a run
  // of tiles, eight tiles of weight rows wide, so that its L2 holds what they
  // share
  const int tiles = a.tiles_m * a.tiles_n, total = tiles * a.splits, per = (total + 7) / 8;
  const int t0 = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (t0 >= min(total, ((int)(blockIdx.x & 7) + 1) * per)) return;
  const int split = t0 / tiles, t = t0 - split * tiles;
  const int sup = t / (8 * a.tiles_m), rest = t - sup * 8 * a.tiles_m;
  const int wide = min(8, a.tiles_n - 8 * sup);
  const int tm = rest / wide, tn = 8 * sup + rest - tm * wide;
  // blocks of 32 rows of X, spread over the tiles evenly
  const int blocks = (int)((a.M + 31) / 32), each = blocks / a.tiles_m, more = blocks % a.tiles_m;
  const int64_t m0 = 32 * ((int64_t)tm * each + min(tm, more)), c0 = (int64_t)tn * tile_n(WIDE);
  const int n = each + (tm < more ? 1 : 0);
  if constexpr (!WIDE) {
    if (n == 8) return tile_product<8, G, GATED, WIDE>(a, lds, m0, c0, split);
    if (n == 7) return tile_product<7, G, GATED, WIDE>(a, lds, m0, c0, split);
    if (n == 6) return tile_product<6, G, GATED, WIDE>(a, lds, m0, c0, split);
    if (n == 5) return tile_product<5, G, GATED, WIDE>(a, lds, m0, c0, split);
  }
  if (n == 4) return tile_product<4, G, GATED, WIDE>(a, lds, m0, c0, split);
  if (n == 3) return tile_product<3, G, GATED, WIDE>(a, lds, m0, c0, split);
  if (n == 2) return tile_product<2, G, GATED, WIDE>(a, lds, m0, c0, split);
  tile_product<1, G, GATED, WIDE>(a, lds, m0, c0, split);
}

template <bool GATED, bool WIDE>
hipError_t tiles_launch(const Args& a, int G, hipStream_t stream) {
  const dim3 grid((unsigned)(8 * ceil_div((int64_t)a.tiles_m * a.tiles_n * a.splits, 8)));
  switch (G) {
    case 32: hipLaunchKernelGGL((linear_kernel<32, GATED, WIDE>), grid, dim3(256), 0, stream, a); break;
    case 64: hipLaunchKernelGGL((linear_kernel<64, GATED, WIDE>), grid, dim3(256), 0, stream, a); break;
    case 128: hipLaunchKernelGGL((linear_kernel<128, GATED, WIDE>), grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL((linear_kernel<0, GATED, WIDE>), grid, dim3(256), 0, stream, a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  return join_finish_launch<GATED>(a.part, a.M, a.N, a.splits, a.e, Terms{}, stream);
}

}  // namespace

size_t linear_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size, bool gated) {
  if (few_tokens(m, d_out, d_in, group_size))
    return linear_vec_workspace(m, d_out, d_in, group_size, gated);
  return plan_for(m, d_out, d_in, group_size, gated).bytes;
}

hipError_t linear_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                         const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                         int64_t d_in, int group_size, bool gated, const Epilogue& e, void* ws,
                         hipStream_t stream) {
  if (few_tokens(m, d_out, d_in, group_size))
    return linear_vec_launch(X, m, ldx, qweight, scales_f16, zeros_f16, d_out, d_in, group_size,
                             gated, e, ws, stream);
  const Plan p = plan_for(m, d_out, d_in, group_size, gated);
  Args a;
  a.x = (const char*)X, a.ldx = 2 * ldx, a.q = qweight, a.s16 = scales_f16, a.z16 = zeros_f16;
  a.part = p.splits > 1 ? (float*)((char*)ws + p.part_off) : nullptr;
  a.e = e, a.M = m, a.N = (int)d_out, a.K = (int)d_in;
  a.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
  a.tiles_m = p.tiles_m, a.tiles_n = p.tiles_n, a.splits = p.splits, a.per_split = p.per_split;
  a.wide = nullptr, a.scales = nullptr, a.cols = 0;
  const int G = group_size == -1 ? 0 : group_size;
  if (!p.wide)
    return gated ? tiles_launch<true, false>(a, G, stream) : tiles_launch<false, false>(a, G, stream);
  const Wide w = wide_of(d_out, d_in, group_size, gated);
  a.wide = (const char*)ws, a.scales = (const float*)((char*)ws + w.scales), a.cols = w.cols;
  const dim3 grid((unsigned)ceil_div(w.cols * (2 * w.nch + w.ng), 256));
  const auto widen = gated ? widen_kernel<true> : widen_kernel<false>;
  hipLaunchKernelGGL(widen, grid, dim3(256), 0, stream, w, e.F, (int)d_in,
                     G == 0 ? (int)d_in : G, qweight, scales_f16, a.z16, (char*)ws);
  const hipError_t st = hipGetLastError();
  if (st != hipSuccess) return st;
  return gated ? tiles_launch<true, true>(a, G, stream) : tiles_launch<false, true>(a, G, stream);
}

}  // namespace gptq
