// Product of the packed 4-bit weights with 8-bit activations (W4A8):
//   Y[i][n] = sx[i] sum_g s[n][g] sum_{k in g} X[i][k] (q[n][k] - z[n][g])
//
// Few tokens: w4_dot.h and w4_vec.h.  More: q - z, within int8, multiplies X on
// the matrix cores, a group's sum an exact 32-bit integer; every group ends with
// two vector operations per sum (to float32, times s into the total), shared by
// nothing: with groups of 128 they take the vector units about as long as the
// products take the matrix cores, with 64 twice as long, with 32 four times.  So
// one group's products run while the one before it is scaled, and what else the
// vector units do is kept small: codes are taken apart by masks, four to an
// operation, once for all rows of X (the four waves of a workgroup stand side by
// side along the weight rows), zeros are taken off four at a time, and X and the
// scales are laid out before (w4a8_layout_kernel), so that both come by direct
// loads and need no further work.
// 8192 tokens through 28672 x 8192, groups of 128: 2.14 ms, 1.80 POP/s, calls
// back to back and the layout's 28 us included (1.86 ms, 2.07 POP/s with one
// group per row; a library int8 product of 8192^3 reaches 2.08; 2.04 ms on
// another card, and launches apart under a tracer 2.18 to 2.36), the vector units busy 75% of the cycles and the matrix cores 48%, at the
// 1.7 GHz that the chip's power allows.  515 tokens through 11008 x 4096, groups
// of 64: 58 us.
// Tried and slower or no faster: three buffers (515 tokens 59 -> 61 us), the
// next chunk's codes taken apart ahead (2048 tokens through 11008 x 4096: 161 ->
// 171), two by two waves, eight waves on 256 x 256 (2.36 -> 2.34 ms), scales as
// halves in mixed operations (4 to 7% slower).
#include "common.h"
#include "kernels.h"
#include "w4_dot.h"

#include <algorithm>

namespace gptq {

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;

constexpr int KCH = 128;           // k per chunk (bytes of a row of X, twice those of a weight row)

// Up to here the kernels for a few tokens, past it the tiles below, whose two
// or three launches have to pay (48 tokens through 11008 x 4096: 13.9 and 23.1
// us; through 28672 x 8192: 64 and 48 us; 64 tokens through 4096 x 4096: 8.4
// and 13.8 us, through 8192 x 8192: 25.0 and 21.4 us).
bool few_tokens(int64_t m, int64_t d_out, int64_t d_in) {
  return m <= 32 || (m <= 64 && d_out * d_in < 60000000);
}

constexpr int PANEL = 32 * KCH;    // bytes of a panel: 32 rows of one chunk

// Where the product's tiles are in the workspace: X as panels of 32 rows by
// 128 columns, and per group and weight row a word with the scale's binary16
// bits below and 128 - zero above.
struct Layout {
  int nch;        // chunks, ceil(d_in / 128)
  int64_t rows;   // rows of X, padded to whole tiles
  int64_t cols;   // weight rows, padded to whole tiles
  int ng;         // groups
  size_t sz_off;  // byte offset of the scales and zeros
  size_t bytes;
};

Layout layout_of(int64_t m, int64_t d_out, int64_t d_in, int group_size, int tm, int tn) {
  Layout l;
  l.nch = (int)ceil_div(d_in, KCH);
  l.rows = ceil_div(m, tm) * tm;
  l.cols = ceil_div(d_out, tn) * tn;
  l.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
  l.sz_off = (size_t)l.rows * l.nch * KCH;
  l.bytes = l.sz_off + (size_t)l.ng * l.cols * 4;
  return l;
}

// The matrix cores take 16 consecutive k per lane.  A word's codes come apart
// as its even and its odd ones (two masks), so X's bytes are put in the same
// order once: 0 2 4 6 1 3 5 7 within every eight.  A panel's 16-byte units are
// stored so that 16 rows read at the same unit fall on different LDS banks.
// Rows past m and columns past d_in are zeros: they add nothing to any sum.
// (8192 x 8192 and 28672 x 64 parameters: 29 us; 515 x 4096: 7.5, mostly a
// launch and the parameters' reads, short pieces of long rows.)
__global__ __launch_bounds__(256) void w4a8_layout_kernel(
    const int8_t* __restrict__ X, int64_t ldx, int64_t M, int N, int K, Layout l,
    const uint16_t* __restrict__ S16, const uint16_t* __restrict__ Z16, int vec,
    char* __restrict__ ws) {
  const int64_t units = l.rows * l.nch * (KCH / 16);
  const int64_t params = ceil_div(l.ng, vec) * l.cols;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < units + params;
       t += (int64_t)gridDim.x * 256) {
    if (t < units) {
      const int upr = l.nch * (KCH / 16);
      const int64_t row = t / upr;
      const int u = (int)(t - row * upr);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (row < M && 16 * u < K) v = *(const uint4*)(X + row * ldx + 16 * u);
      uint4 o;
      o.x = __builtin_amdgcn_perm(v.y, v.x, 0x06040200u);
      o.y = __builtin_amdgcn_perm(v.y, v.x, 0x07050301u);
      o.z = __builtin_amdgcn_perm(v.w, v.z, 0x06040200u);
      o.w = __builtin_amdgcn_perm(v.w, v.z, 0x07050301u);
      const int r = (int)(row & 31), c = u >> 3, uu = (u & 7) ^ ((r >> 1) & 7);
      *(uint4*)(ws + ((row >> 5) * l.nch + c) * PANEL + r * KCH + 16 * uu) = o;
    } else {
      // a weight row's parameters of `vec` groups (what its alignment allows
      // in one load); neighbouring threads take neighbouring rows, so that the
      // groups' planes are written whole
      const int64_t p = t - units;
      const int g = (int)(p / l.cols) * vec;
      const int64_t n = p % l.cols;
      uint16_t s[8], z[8];
      if (n < N) {
        const int64_t at = n * l.ng + g;
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
      uint32_t* out = (uint32_t*)(ws + l.sz_off) + (int64_t)g * l.cols + n;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= vec) break;
        out[i * l.cols] =
            n < N ? s[i] | (uint32_t)(128 - (Z16 ? w4vec::whole_zero(z[i]) : 8)) << 16 : 0u;
      }
    }
  }
}

// Direct global -> LDS load of 16 bytes per lane: lane l's bytes land at
// lds_off + 16 l.  In asm, since the compiler would wait for every load in
// flight before any LDS read; the loop waits for them itself.
__device__ __forceinline__ void dma16(const void* base, uint32_t voff, uint32_t lds_off) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const uint32_t blo = __builtin_amdgcn_readfirstlane((uint32_t)b);
  const uint32_t bhi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  const void* sbase = (const void*)(uintptr_t)(((uint64_t)bhi << 32) | blo);
  const uint32_t lbase = __builtin_amdgcn_readfirstlane(lds_off);
  __asm__ volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                   :
                   : "v"(voff), "s"(sbase), "s"(lbase)
                   : "memory", "m0");
}

// q - z of a word's codes as int8: the even codes, then the odd ones.  Each
// byte is q + (128 - z), which stays within 0..255 for |z| <= 100, so no
// carry crosses bytes; flipping the top bit takes the 128 off again.
__device__ __forceinline__ void minus_zero(uint32_t w, uint32_t zc, int& even, int& odd) {
  even = (int)(((w & 0x0f0f0f0fu) + zc) ^ 0x80808080u);
  odd = (int)((((w >> 4) & 0x0f0f0f0fu) + zc) ^ 0x80808080u);
}

struct MulArgs {
  const char* ws;
  const float* sx;
  const uint32_t* q;
  float* y;       // Y, or the splits' partial products
  Layout l;
  int64_t M;
  int N;
  int row_bytes;  // of a packed weight row
  int tiles_m, tiles_n;
  int splits, per_split;  // of the chunks
};

template <int MI, int NI, int G>
struct Shape {
  static constexpr int TM = 32 * MI, TN = 128 * NI;
  static constexpr int GPC = G == 0 ? 0 : KCH / G;  // groups per chunk
  static constexpr int ABYTES = TM * KCH, BBYTES = TN * (KCH / 2), SZBYTES = GPC * TN * 4;
  static constexpr int STAGE = ABYTES + BBYTES + SZBYTES;
};

// Four waves side by side, each 32 MI rows of X by 32 NI weight rows: a wave
// takes the codes of its own weight rows apart, and none twice.  G: group
// size, 0 for one group per row.
template <int MI, int NI, int G>
__device__ __forceinline__ void tile_product(const MulArgs& a, char* lds, int64_t m0, int n0,
                                             int split) {
  typedef Shape<MI, NI, G> S;
  constexpr int TN = S::TN, GPC = S::GPC, ABYTES = S::ABYTES, BBYTES = S::BBYTES;
  constexpr int STAGE = S::STAGE;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, l32 = lane & 31;
  const int nch = a.l.nch, c0 = split * a.per_split, c1 = min(nch, c0 + a.per_split);

  // direct loads: X panels and group words are copied as they are; a weight
  // row's 64 bytes of a chunk go to units that put 16 rows on different banks
  const char* xbase = a.ws + (m0 >> 5) * nch * PANEL;
  const char* qbase = (const char*)a.q + (int64_t)n0 * a.row_bytes;
  const uint32_t* sz = (const uint32_t*)(a.ws + a.l.sz_off) + n0 + 32 * NI * wave;
  uint32_t qrow[2 * NI];
#pragma unroll
  for (int j = 0; j < 2 * NI; ++j)
    qrow[j] = (uint32_t)min(16 * (2 * NI * wave + j) + (lane >> 2), a.N - 1 - n0) * a.row_bytes;
  const uint32_t qu = 16 * ((lane & 3) ^ ((lane >> 4) & 3));
  auto issue = [&](int c, int buf) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + buf * STAGE;
#pragma unroll
    for (int j = 0; j < MI; ++j) {  // 1 KB pieces of the tile's MI panels
      const int piece = MI * wave + j;
      dma16(xbase + ((int64_t)(piece >> 2) * nch + c) * PANEL + (piece & 3) * 1024, lane * 16,
            dst + piece * 1024);
    }
    const uint32_t k = min((uint32_t)c * (KCH / 2) + qu, (uint32_t)a.row_bytes - 16);
#pragma unroll
    for (int j = 0; j < 2 * NI; ++j)
      dma16(qbase, qrow[j] + k, dst + ABYTES + (2 * NI * wave + j) * 1024);
    if constexpr (G != 0) {
      if (lane < 8 * NI) {  // this wave's 32 NI words of each group
#pragma unroll
        for (int g = 0; g < GPC; ++g)
          dma16(sz + (int64_t)min(c * GPC + g, a.l.ng - 1) * a.l.cols, lane * 16,
                dst + ABYTES + BBYTES + (g * TN + 32 * NI * wave) * 4);
      }
    }
  };
  // the scale of row threadIdx.x, for the end
  float sx_mine = 1.0f;
  if (a.splits == 1 && threadIdx.x < 32 * MI)
    sx_mine = a.sx[min(m0 + (int64_t)threadIdx.x, a.M - 1)];
  uint32_t row_sz[NI];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) row_sz[ni] = G == 0 ? sz[32 * ni + l32] : 0u;

  constexpr int BL = MI * NI;  // 32 x 32 blocks of a wave, ni the faster index
  f32x16 tot[G == 0 ? 1 : BL];
  i32x16 sum[G == 0 ? BL : 1];
#pragma unroll
  for (int mi = 0; mi < BL; ++mi)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (G == 0)
        sum[mi][i] = 0;
      else
        tot[mi][i] = 0.0f;
    }
  issue(c0, 0);
  for (int c = c0; c < c1; ++c) {
    const int buf = (c - c0) & 1;
    // chunk c has landed, and chunk c - 1's buffer is read
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (c + 1 < c1) issue(c + 1, buf ^ 1);
    const char* la = lds + buf * STAGE;
    const char* lb = lds + buf * STAGE + ABYTES + (32 * NI * wave + l32) * (KCH / 2);
    const uint32_t* lz =
        (const uint32_t*)(lds + buf * STAGE + ABYTES + BBYTES) + 32 * NI * wave + l32;
    const int sw = (l32 >> 2) & 3;
    // MFMA q of a chunk takes, in lane half h, unit u of X: with groups of 32
    // the two halves share 32 consecutive k, otherwise 64
    float scale[NI][GPC ? GPC : 1];
    i32x4 bf[NI][4];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      uint32_t zc[GPC ? GPC : 1];
#pragma unroll
      for (int g = 0; g < (GPC ? GPC : 1); ++g) {
        const uint32_t v = G == 0 ? row_sz[ni] : lz[g * TN + 32 * ni];
        scale[ni][g] = w4vec::half_bits((uint16_t)v);
        zc[g] = __builtin_amdgcn_perm(v, v, 0x02020202u);
        asm("" : "+v"(scale[ni][g]));  // or every product converts it again
      }
      const char* lw = lb + 32 * ni * (KCH / 2);
      uint32_t w[8];
      if constexpr (G == 32) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint2 v = *(const uint2*)(lw + 16 * (q ^ sw) + 8 * h);
          w[2 * q] = v.x, w[2 * q + 1] = v.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 v = *(const uint4*)(lw + 16 * ((2 * j + h) ^ sw));
          w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int o[4];
        minus_zero(w[2 * q], zc[q * GPC / 4], o[0], o[1]);
        minus_zero(w[2 * q + 1], zc[q * GPC / 4], o[2], o[3]);
        bf[ni][q] = i32x4{o[0], o[1], o[2], o[3]};
      }
    }
    auto xfrag = [&](int mi, int q) __attribute__((always_inline)) {
      const int u = G == 32 ? 2 * q + h : 4 * (q >> 1) + 2 * h + (q & 1);
      return *(const i32x4*)(la + mi * PANEL + l32 * KCH + 16 * (u ^ ((l32 >> 1) & 7)));
    };
    if constexpr (G == 0) {
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const i32x4 x = xfrag(mi, q);
#pragma unroll
          for (int ni = 0; ni < NI; ++ni)
            sum[mi * NI + ni] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, bf[ni][q],
                                                                      sum[mi * NI + ni], 0, 0, 0);
        }
    } else {
      // step s multiplies for one block and one group while the step before it
      // is scaled into its total; the steps of 32 rows follow one another
      constexpr int PER = NI * GPC, STEPS = MI * PER, QPS = 4 / GPC;
      i32x4 af[2][4];
      i32x16 acc[2];
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
          acc[s & 1] = i32x16{};
#pragma unroll
          for (int q = 0; q < QPS; ++q)
            acc[s & 1] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
                af[mi & 1][g * QPS + q], bf[ni][g * QPS + q], acc[s & 1], 0, 0, 0);
        }
        if (s > 0) {
          const int p = s - 1;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            tot[p / GPC][i] = fmaf(scale[p % PER / GPC][p % GPC], (float)acc[p & 1][i], tot[p / GPC][i]);
        }
#pragma unroll
        for (int q = 0; q < QPS; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);        // an LDS read
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);        // a product
          __builtin_amdgcn_sched_group_barrier(0x002, 32 / QPS, 0); // its share of the scaling
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // The rows' scales by way of LDS: read where they are used, each row's store
  // waited for its load (12 us of every workgroup's time).
  __syncthreads();
  float* const ls = (float*)lds;
  if (threadIdx.x < 32 * MI) ls[threadIdx.x] = sx_mine;
  __syncthreads();
  float* const y = a.y + (int64_t)split * a.M * a.N + m0 * a.N + n0;
  const int rows = (int)min((int64_t)(32 * MI), a.M - m0);
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int r0 = 32 * mi + 2 * i + 4 * h;
      const float4 sx4 = *(const float4*)(ls + r0);
      const float sx[4] = {sx4.x, sx4.y, sx4.z, sx4.w};
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        const int col = 32 * (NI * wave + ni) + l32;
        const bool in = n0 + col < a.N;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v;
          if constexpr (G == 0)
            v = w4vec::half_bits((uint16_t)row_sz[ni]) * (float)sum[mi * NI + ni][i + e];
          else
            v = tot[mi * NI + ni][i + e];
          if (in && r0 + e < rows) y[(int64_t)(r0 + e) * a.N + col] = sx[e] * v;
        }
      }
    }
}

template <int MI, int NI, int G>
__global__ __launch_bounds__(256, 2) void w4a8_kernel(MulArgs a) {
  constexpr int TM = 32 * MI, TN = 128 * NI;
  __shared__ __attribute__((aligned(1024))) char lds[2 * Shape<MI, NI, G>::STAGE];
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
  const int64_t m0 = (int64_t)tm * TM;
  const int n0 = tn * TN;
  // the last rows' tile does the work of the rows that are there
  const int64_t left = a.M - m0;
  if constexpr (MI >= 2) {
    if (left <= 32) return tile_product<1, NI, G>(a, lds, m0, n0, split);
  }
  if constexpr (MI >= 3) {
    if (left <= 64) return tile_product<2, NI, G>(a, lds, m0, n0, split);
  }
  if constexpr (MI >= 4) {
    if (left <= 96) return tile_product<3, NI, G>(a, lds, m0, n0, split);
  }
  tile_product<MI, NI, G>(a, lds, m0, n0, split);
}

struct Plan {
  int mi, ni;  // tile: 32 mi rows of X by 128 ni weight rows
  int splits, per_split;
  Layout l;
  size_t part_off, bytes;
};

// Tiles of 128 x 256 (X by weight rows) where they fill rounds of two per CU;
// else 128, 96, 64 or 32 rows of X by 128, and k over several workgroups, by
// the least of a time in us: workgroups share a CU, a tile takes `alone` by
// itself and no CU does better than one per `shared` (each measured at 32
// chunks of groups of 128); splits add a launch and their sums' bytes at some
// 4 TB/s.  4096 columns through 4096 weight rows: 2048 tokens take 56 us with
// 128 rows, 57 with 96 and 60 with 64; 1024 tokens 36, 41 and 34; 256 tokens
// 23.3 us with 32 rows in one piece, 21.2 in two.  1500 tokens through 4096 x
// 11008 in groups of 64: 142, 127 and 133 us with 128, 96 and 64.
Plan plan_for(int64_t m, int64_t d_out, int64_t d_in, int group_size) {
  constexpr double shared[4] = {9.5, 14.0, 19.5, 25.0}, alone[4] = {18.0, 25.0, 31.0, 38.0};
  Plan p;
  const int nch = (int)ceil_div(d_in, KCH);
  const int64_t wide = ceil_div(m, 128) * ceil_div(d_out, 256);
  p.mi = 4, p.ni = 2;
  int64_t splits = 1;
  if (10 * wide < 9 * 512 * ceil_div(wide, 512)) {
    p.ni = 1;
    double best = 0.0;
    for (int s = 1; s <= 16 && (s == 1 || s <= nch / 2); s *= 2)
      for (int i = 0; i < 4; ++i) {
        const int64_t n = ceil_div(m, 32 * (i + 1)) * ceil_div(d_out, 128) * s;
        double us = std::max((double)ceil_div(n, 256) * shared[i], alone[i]) * nch / 32 / s;
        if (s > 1) us += 3.0 + 1e-6 * (double)(m * d_out) * (s + 1);
        if (best == 0.0 || us < best) best = us, p.mi = i + 1, splits = s;
      }
  }
  p.per_split = (int)ceil_div(nch, splits);
  p.splits = (int)ceil_div(nch, p.per_split);
  p.l = layout_of(m, d_out, d_in, group_size, 32 * p.mi, 128 * p.ni);
  p.part_off = (p.l.bytes + 255) / 256 * 256;
  p.bytes = p.splits > 1 ? p.part_off + (size_t)p.splits * m * d_out * 4 : p.l.bytes;
  return p;
}

template <int MI, int NI>
void launch(const MulArgs& a, int G, hipStream_t stream) {
  const dim3 grid((unsigned)(8 * ceil_div((int64_t)a.tiles_m * a.tiles_n * a.splits, 8)));
  switch (G) {
    case 32: hipLaunchKernelGGL((w4a8_kernel<MI, NI, 32>), grid, dim3(256), 0, stream, a); break;
    case 64: hipLaunchKernelGGL((w4a8_kernel<MI, NI, 64>), grid, dim3(256), 0, stream, a); break;
    case 128: hipLaunchKernelGGL((w4a8_kernel<MI, NI, 128>), grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL((w4a8_kernel<MI, NI, 0>), grid, dim3(256), 0, stream, a);
  }
}

}  // namespace

size_t w4a8_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size) {
  if (!few_tokens(m, d_out, d_in)) return plan_for(m, d_out, d_in, group_size).bytes;
  const int G = group_size == -1 ? 0 : group_size;
  return w4vec::dot_takes(m, d_in) ? 0 : w4vec::vec_plan(true, m, d_out, d_in, G).ws_bytes;
}

hipError_t w4a8_launch(const int8_t* X, const float* x_scales, int64_t m, int64_t ldx,
                       const uint32_t* qweight, const uint16_t* scales_f16,
                       const uint16_t* zeros_f16, int64_t d_out, int64_t d_in, int group_size,
                       float* Y, void* ws, hipStream_t stream) {
  const int G = group_size == -1 ? 0 : group_size;
  if (few_tokens(m, d_out, d_in)) {
    w4vec::VecArgs v;
    v.x = (const char*)X, v.sx = x_scales, v.q = qweight, v.s16 = scales_f16, v.z16 = zeros_f16;
    v.y = Y, v.ldx = ldx, v.m = (int)m, v.n = (int)d_out, v.k = (int)d_in;
    v.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
    v.vec = w4vec::scale_vec(scales_f16, zeros_f16, v.ng);
    return w4vec::dot_takes(m, d_in) ? w4vec::dot_launch<true>(v, G, stream)
                                     : w4vec::vec_launch<true>(v, G, ws, stream);
  }
  const Plan p = plan_for(m, d_out, d_in, group_size);
  const int vec = w4vec::scale_vec(scales_f16, zeros_f16, p.l.ng);
  const int64_t items = p.l.rows * p.l.nch * (KCH / 16) + (int64_t)ceil_div(p.l.ng, vec) * p.l.cols;
  hipLaunchKernelGGL(w4a8_layout_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(items, 256), 8192)),
                     dim3(256), 0, stream, X, ldx, m, (int)d_out, (int)d_in, p.l, scales_f16,
                     zeros_f16, vec, (char*)ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  MulArgs a;
  a.ws = (const char*)ws, a.sx = x_scales, a.q = qweight, a.l = p.l, a.M = m;
  a.y = p.splits > 1 ? (float*)((char*)ws + p.part_off) : Y;
  a.N = (int)d_out, a.row_bytes = (int)(d_in / 2);
  a.tiles_m = (int)(p.l.rows / (32 * p.mi)), a.tiles_n = (int)(p.l.cols / (128 * p.ni));
  a.splits = p.splits, a.per_split = p.per_split;
  switch (p.mi) {
    case 4: p.ni == 2 ? launch<4, 2>(a, G, stream) : launch<4, 1>(a, G, stream); break;
    case 3: launch<3, 1>(a, G, stream); break;
    case 2: launch<2, 1>(a, G, stream); break;
    default: launch<1, 1>(a, G, stream);
  }
  e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  return w4vec::join_launch(a.y, x_scales, m, (int)d_out, p.splits, Y, stream);
}

}  // namespace gptq
