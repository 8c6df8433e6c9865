// The W4A16 product with its epilogue, for more than a few tokens:
//   Y = act(X W_hat^T + bias) + residual, or gated by pairs of weight rows
//   (linear_epi.h), W_hat[n][k] = s[n][k/g] (q[n][k] - z[n][k/g]).
//
// q - z is exact in bf16, so products with X are exact in float32; a group's sum
// stands by itself and is scaled into the total with one operation per sum.
#include "common.h"
#include "kernels.h"
#include "w4_dot.h"

#include <algorithm>

namespace gptq {

namespace {

constexpr int KCH = 64;  // k per chunk: 128 bytes of a row of X, 32 of a weight row

// Per group and weight row a word with the scale's binary16 bits below and the
// zero's above.  Columns stand in the order in which the tiles take weight rows:
// gated, 32 gate rows, then the 32 up rows that go with them.
struct Layout {
  int64_t cols;  // weight rows, padded to whole tiles
  int ng;
  size_t bytes;
};

template <bool GATED>
__device__ __forceinline__ int64_t weight_row(int64_t c, int F) {
  return GATED ? (c >> 6) * 32 + (c & 31) + ((c >> 5) & 1) * F : c;
}
template <bool GATED>
__device__ __forceinline__ bool weight_row_in(int64_t c, int F) {
  return GATED ? (c >> 6) * 32 + (c & 31) < F : c < F;
}

template <bool GATED>
__global__ __launch_bounds__(256) void linear_layout_kernel(Layout l, int F,
                                                            const uint16_t* __restrict__ S16,
                                                            const uint16_t* __restrict__ Z16,
                                                            int vec, uint32_t* __restrict__ ws) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t params = ceil_div(l.ng, vec) * l.cols;
  if (t >= params) return;
  const int g = (int)(t / l.cols) * vec;
  const int64_t c = t % l.cols;
  const bool in = weight_row_in<GATED>(c, F);
  uint16_t s[8] = {}, z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = 0x4800;  // 8
  if (in) {
    const int64_t at = weight_row<GATED>(c, F) * l.ng + g;
    if (vec == 8) {
      *(uint4*)s = *(const uint4*)(S16 + at);
      if (Z16) *(uint4*)z = *(const uint4*)(Z16 + at);
    } else if (vec == 4) {
      *(uint2*)s = *(const uint2*)(S16 + at);
      if (Z16) *(uint2*)z = *(const uint2*)(Z16 + at);
    } else if (vec == 2) {
      *(uint32_t*)s = *(const uint32_t*)(S16 + at);
      if (Z16) *(uint32_t*)z = *(const uint32_t*)(Z16 + at);
    } else {
      s[0] = S16[at];
      if (Z16) z[0] = Z16[at];
    }
  }
  uint32_t* out = ws + (int64_t)g * l.cols + c;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < vec) out[i * l.cols] = (uint32_t)s[i] | (uint32_t)z[i] << 16;
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

struct Args {
  const char* x;
  int64_t ldx;    // bytes
  const uint32_t* q;
  const uint32_t* sz;
  float* part;    // splits' sums [splits][M][N], null: finished here
  Epilogue e;
  Layout l;
  int64_t M;
  int N, K;
  int tiles_m, tiles_n;
  int splits, per_split;  // of the chunks
};

template <int MI, int NI, int G>
struct Shape {
  static constexpr int TM = 32 * MI, TN = 128 * NI;
  static constexpr int GPC = G == 0 ? 0 : G >= KCH ? 1 : KCH / G;  // groups in a chunk
  static constexpr int ABYTES = TM * 2 * KCH, BBYTES = TN * (KCH / 2), SZBYTES = GPC * TN * 4;
  static constexpr int STAGE = ABYTES + BBYTES + SZBYTES;
  static constexpr int OUT = 32 * TN * 4;  // 32 rows of sums on their way out
  static constexpr int LDS = 2 * STAGE > OUT ? 2 * STAGE : OUT;
};

// Four waves side by side, each 32 MI rows of X by 32 NI weight rows: a wave
// takes the codes of its own weight rows apart, and none twice.  G: group size,
// 0 for one group per row.  GATED: NI is 2, gate rows and up rows.
template <int MI, int NI, int G, bool GATED>
__device__ __forceinline__ void tile_product(const Args& a, char* lds, int64_t m0, int64_t c0,
                                             int split) {
  typedef Shape<MI, NI, G> S;
  constexpr int TN = S::TN, GPC = S::GPC, ABYTES = S::ABYTES, BBYTES = S::BBYTES;
  constexpr int STAGE = S::STAGE;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, l32 = lane & 31;
  const int nch = (a.K + KCH - 1) / KCH, ch0 = split * a.per_split,
            ch1 = min(nch, ch0 + a.per_split);
  const int64_t wcol = c0 + 32 * NI * wave;  // this wave's first column
  const int F = a.e.F;

  // direct loads, 1 KB each: 8 rows of X, or 32 weight rows, at units that put
  // 16 rows on different banks
  const char* xrow[MI];
#pragma unroll
  for (int j = 0; j < MI; ++j)
    xrow[j] = a.x + min(m0 + 8 * (MI * wave + j) + (lane >> 3), a.M - 1) * a.ldx;
  int xu[MI];
#pragma unroll
  for (int j = 0; j < MI; ++j)
    xu[j] = 16 * ((lane & 7) ^ (((8 * (MI * wave + j) + (lane >> 3)) >> 1) & 7));
  const char* qrow[NI];
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int64_t c = wcol + 32 * j + (lane >> 1);
    qrow[j] = (const char*)a.q +
              (weight_row_in<GATED>(c, F) ? weight_row<GATED>(c, F) : 0) * (a.K / 2);
  }
  const int qu = 16 * ((lane & 1) ^ ((lane >> 4) & 1));
  const uint32_t* sz = a.sz + wcol + 4 * lane;
  auto issue = [&](int c, int buf) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + buf * STAGE;
#pragma unroll
    for (int j = 0; j < MI; ++j)
      w4vec::dma16_at(xrow[j] + min(c * 2 * KCH + xu[j], 2 * a.K - 16),
                      dst + (MI * wave + j) * 1024);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      w4vec::dma16_at(qrow[j] + min(c * (KCH / 2) + qu, a.K / 2 - 16),
                      dst + ABYTES + (NI * wave + j) * 1024);
    if constexpr (G != 0) {
      if (lane < 8 * NI) {  // this wave's 32 NI words of each group
#pragma unroll
        for (int g = 0; g < GPC; ++g)
          w4vec::dma16_at(sz + (int64_t)min(G >= KCH ? c * KCH / G : c * GPC + g, a.l.ng - 1) * a.l.cols,
                          dst + ABYTES + BBYTES + (g * TN + 32 * NI * wave) * 4);
      }
    }
  };
  uint32_t row_sz[NI];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) row_sz[ni] = G == 0 ? a.sz[wcol + 32 * ni + l32] : 0u;

  constexpr int BL = MI * NI;  // 32 x 32 blocks of a wave, ni the faster index
  f32x16 tot[BL];
#pragma unroll
  for (int b = 0; b < BL; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) tot[b][i] = 0.0f;
  issue(ch0, 0);
  for (int c = ch0; c < ch1; ++c) {
    const int buf = (c - ch0) & 1;
    // chunk c has landed, and chunk c - 1's buffer is read
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (c + 1 < ch1) issue(c + 1, buf ^ 1);
    const char* la = lds + buf * STAGE + l32 * 2 * KCH;
    const char* lb = lds + buf * STAGE + ABYTES + (32 * NI * wave + l32) * (KCH / 2);
    const uint32_t* lz =
        (const uint32_t*)(lds + buf * STAGE + ABYTES + BBYTES) + 32 * NI * wave + l32;
    const int sw = (l32 >> 3) & 1;
    // MFMA q of a chunk takes, in lane half h, unit u of X: with groups of 32
    // the two halves share 32 consecutive k, otherwise 64
    auto unit = [&](int q) __attribute__((always_inline)) {
      return G == 32 ? 4 * (q >> 1) + 2 * h + (q & 1) : 4 * h + q;
    };
    const bool tail = (c + 1) * KCH > a.K;  // past the row's end: zeros
    float scale[NI][GPC ? GPC : 1];
    bf16x8 bf[NI][4];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      float z[GPC ? GPC : 1];
#pragma unroll
      for (int g = 0; g < (GPC ? GPC : 1); ++g) {
        const uint32_t v = G == 0 ? row_sz[ni] : lz[g * TN + 32 * ni];
        scale[ni][g] = w4vec::half_bits((uint16_t)v);
        z[g] = w4vec::half_bits((uint16_t)(v >> 16));
        asm("" : "+v"(scale[ni][g]), "+v"(z[g]));  // or every product converts it again
      }
      const char* lw = lb + 32 * ni * (KCH / 2);
      uint32_t w[4];
      if constexpr (G == 32) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint2 v = *(const uint2*)(lw + 16 * (j ^ sw) + 8 * h);
          w[2 * j] = v.x, w[2 * j + 1] = v.y;
        }
      } else {
        const uint4 v = *(const uint4*)(lw + 16 * (h ^ sw));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bf[ni][q] = minus_zero(w[q], z[G == 32 ? q >> 1 : 0]);
        if (tail && c * KCH + 8 * unit(q) >= a.K) bf[ni][q] = bf16x8{};
      }
    }
    auto xfrag = [&](int mi, int q) __attribute__((always_inline)) {
      return *(const bf16x8*)(la + mi * 32 * 2 * KCH + 16 * (unit(q) ^ ((l32 >> 1) & 7)));
    };
    if constexpr (G == 0) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8 x = xfrag(mi, q);
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            tot[mi * NI + ni] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, bf[ni][q],
                                                                        tot[mi * NI + ni], 0, 0, 0);
        }
    } else {
      // step s multiplies for one block and one group while the step before it
      // is scaled into its total; the steps of 32 rows follow one another
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
                af[mi & 1][g * QPS + q], bf[ni][g * QPS + q], acc[s & 1], 0, 0, 0);
        }
        if (s > 0) {
          const int p = s - 1;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            tot[p / GPC][i] = fmaf(scale[p % PER / GPC][p % GPC], acc[p & 1][i], tot[p / GPC][i]);
        }
#pragma unroll
        for (int q = 0; q < QPS; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);        // an LDS read
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);        // a product
          __builtin_amdgcn_sched_group_barrier(0x002, 16 / QPS, 0); // its share of the scaling
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (G == 0) {
#pragma unroll
    for (int b = 0; b < BL; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) tot[b][i] *= w4vec::half_bits((uint16_t)row_sz[b % NI]);
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
#pragma unroll 1
  for (int mi = 0; mi < MI; ++mi) {
    __syncthreads();
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
    __syncthreads();
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
      if (a.part) {
        float* o = a.part + ((int64_t)split * a.M + row) * a.N + u0 + col;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < ncol) {
            o[i] = v0[i];
            if constexpr (GATED) o[F + i] = v1[i];
          }
      } else {
        finish4<GATED>(a.e, row, u0 + col, ncol, v0, v1);
      }
    }
  }
}

template <int MI, int NI, int G, bool GATED>
__global__ __launch_bounds__(256, 2) void linear_kernel(Args a) {
  constexpr int TM = 32 * MI, TN = 128 * NI;
  __shared__ __attribute__((aligned(1024))) char lds[Shape<MI, NI, G>::LDS];
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
  const int64_t m0 = (int64_t)tm * TM, c0 = (int64_t)tn * TN;
  // the last rows' tile does the work of the rows that are there
  const int64_t left = a.M - m0;
  if constexpr (MI >= 2) {
    if (left <= 32) return tile_product<1, NI, G, GATED>(a, lds, m0, c0, split);
  }
  if constexpr (MI >= 4) {
    if (left <= 64) return tile_product<2, NI, G, GATED>(a, lds, m0, c0, split);
  }
  tile_product<MI, NI, G, GATED>(a, lds, m0, c0, split);
}

// Few tokens: the kernels that read the weights once for all of them.
bool few_tokens(int64_t m) { return m <= 64; }

struct Plan {
  int mi, ni;  // tile: 32 mi rows of X by 128 ni weight rows
  int splits, per_split;
  Layout l;
  size_t part_off, bytes;
};

Plan plan_for(int64_t m, int64_t d_out, int64_t d_in, int group_size, bool gated) {
  Plan p;
  const int nch = (int)ceil_div(d_in, KCH);
  p.mi = 4, p.ni = gated || ceil_div(m, 128) * ceil_div(d_out, 256) >= 256 ? 2 : 1;
  while (p.mi > 1 && ceil_div(m, 32 * p.mi) * ceil_div(d_out, 128 * p.ni) < 256) p.mi /= 2;
  int64_t splits = 1;
  while (splits < 8 && splits * 8 <= nch &&
         ceil_div(m, 32 * p.mi) * ceil_div(d_out, 128 * p.ni) * splits < 256)
    splits *= 2;
  p.per_split = (int)ceil_div(nch, splits);
  p.splits = (int)ceil_div(nch, p.per_split);
  p.l.cols = ceil_div(gated ? d_out / 2 : d_out, (gated ? 64 : 128) * p.ni) * 128 * p.ni;
  p.l.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
  p.l.bytes = (size_t)p.l.ng * p.l.cols * 4;
  p.part_off = (p.l.bytes + 255) / 256 * 256;
  p.bytes = p.splits > 1 ? p.part_off + (size_t)p.splits * m * d_out * 4 : p.l.bytes;
  return p;
}

template <int MI, int NI, bool GATED>
void launch(const Args& a, int G, hipStream_t stream) {
  const dim3 grid((unsigned)(8 * ceil_div((int64_t)a.tiles_m * a.tiles_n * a.splits, 8)));
  switch (G) {
    case 32: hipLaunchKernelGGL((linear_kernel<MI, NI, 32, GATED>), grid, dim3(256), 0, stream, a); break;
    case 64: hipLaunchKernelGGL((linear_kernel<MI, NI, 64, GATED>), grid, dim3(256), 0, stream, a); break;
    case 128: hipLaunchKernelGGL((linear_kernel<MI, NI, 128, GATED>), grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL((linear_kernel<MI, NI, 0, GATED>), grid, dim3(256), 0, stream, a);
  }
}

template <bool GATED>
hipError_t tiles_launch(Args a, const Plan& p, int group_size, const uint16_t* scales_f16,
                        const uint16_t* zeros_f16, void* ws, hipStream_t stream) {
  const int vec = w4vec::scale_vec(scales_f16, zeros_f16, p.l.ng);
  const int64_t items = ceil_div(p.l.ng, vec) * p.l.cols;
  hipLaunchKernelGGL((linear_layout_kernel<GATED>), dim3((unsigned)ceil_div(items, 256)), dim3(256),
                     0, stream, p.l, a.e.F, scales_f16, zeros_f16, vec, (uint32_t*)ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int G = group_size == -1 ? 0 : group_size;
  if constexpr (GATED) {
    switch (p.mi) {
      case 4: launch<4, 2, true>(a, G, stream); break;
      case 2: launch<2, 2, true>(a, G, stream); break;
      default: launch<1, 2, true>(a, G, stream);
    }
  } else {
    switch (p.mi) {
      case 4: p.ni == 2 ? launch<4, 2, false>(a, G, stream) : launch<4, 1, false>(a, G, stream); break;
      case 2: launch<2, 1, false>(a, G, stream); break;
      default: launch<1, 1, false>(a, G, stream);
    }
  }
  e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  return join_finish_launch<GATED>(a.part, a.M, a.N, p.splits, a.e, stream);
}

}  // namespace

size_t linear_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size, bool gated) {
  if (few_tokens(m)) return linear_vec_workspace(m, d_out, d_in, group_size, gated);
  return plan_for(m, d_out, d_in, group_size, gated).bytes;
}

hipError_t linear_launch(const void* X, int64_t m, int64_t ldx, const uint32_t* qweight,
                         const uint16_t* scales_f16, const uint16_t* zeros_f16, int64_t d_out,
                         int64_t d_in, int group_size, bool gated, const Epilogue& e, void* ws,
                         hipStream_t stream) {
  if (few_tokens(m))
    return linear_vec_launch(X, m, ldx, qweight, scales_f16, zeros_f16, d_out, d_in, group_size,
                             gated, e, ws, stream);
  const Plan p = plan_for(m, d_out, d_in, group_size, gated);
  Args a;
  a.x = (const char*)X, a.ldx = 2 * ldx, a.q = qweight, a.sz = (const uint32_t*)ws;
  a.part = p.splits > 1 ? (float*)((char*)ws + p.part_off) : nullptr;
  a.e = e, a.l = p.l, a.M = m, a.N = (int)d_out, a.K = (int)d_in;
  a.tiles_m = (int)ceil_div(m, 32 * p.mi), a.tiles_n = (int)(p.l.cols / (128 * p.ni));
  a.splits = p.splits, a.per_split = p.per_split;
  return gated ? tiles_launch<true>(a, p, group_size, scales_f16, zeros_f16, ws, stream)
               : tiles_launch<false>(a, p, group_size, scales_f16, zeros_f16, ws, stream);
}

}  // namespace gptq
