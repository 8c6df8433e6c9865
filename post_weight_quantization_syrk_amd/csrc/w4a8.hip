// Product of the packed 4-bit weights with 8-bit activations (W4A8):
//   Y[i][n] = sx[i] sum_k X[i][k] s[n][k/g] (q[n][k] - z[n][k/g])
#include "common.h"
#include "kernels.h"
#include "w4_dot.h"

#include <hip/hip_fp16.h>
#include <algorithm>

namespace gptq {

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;

constexpr int KCH = 128;           // k per chunk (bytes of a row of X, twice those of a weight row)
constexpr int VEC_M = 64;          // up to here w4_vec.h's kernel
constexpr int PANEL = 32 * KCH;    // bytes of a panel: 32 rows of one chunk

// Where the product's tiles are in the workspace: X as panels of 32 rows by
// 128 columns, and per group and weight row the scale and the zero.
struct Layout {
  int nch;        // chunks, ceil(d_in / 128)
  int64_t rows;   // rows of X, padded to whole tiles
  int64_t cols;   // weight rows, padded to whole tiles
  int ng;         // groups
  size_t st_off;  // byte offset of the scales
  size_t bytes;
};

struct GroupParam {
  float s;
  uint32_t z;  // 128 - zero in every byte
};

Layout layout_of(int64_t m, int64_t d_out, int64_t d_in, int group_size, int tm, int tn) {
  Layout l;
  l.nch = (int)ceil_div(d_in, KCH);
  l.rows = ceil_div(m, tm) * tm;
  l.cols = ceil_div(d_out, tn) * tn;
  l.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
  l.st_off = (size_t)l.rows * l.nch * KCH;
  l.bytes = l.st_off + (size_t)l.ng * l.cols * sizeof(GroupParam);
  return l;
}

// The matrix cores take 16 consecutive k per lane.  A word's codes come apart
// as its even and its odd ones (two masks), so X's bytes are put in the same
// order once: 0 2 4 6 1 3 5 7 within every eight.  A panel's 16-byte units are
// stored so that 16 rows read at the same unit fall on different LDS banks.
// Rows past m and columns past d_in are zeros: they add nothing to any sum.
__global__ __launch_bounds__(256) void w4a8_layout_kernel(
    const int8_t* __restrict__ X, int64_t ldx, int64_t M, int N, int K, Layout l,
    const uint16_t* __restrict__ S16, const uint16_t* __restrict__ Z16, char* __restrict__ ws) {
  const int64_t units = l.rows * l.nch * (KCH / 16);
  const int64_t params = (int64_t)l.ng * l.cols;
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
      const int64_t p = t - units;
      const int g = (int)(p / l.cols);
      const int64_t n = p - (int64_t)g * l.cols;
      GroupParam gp = {0.0f, 0u};
      if (n < N) {
        gp.s = __half2float(__ushort_as_half(S16[n * l.ng + g]));
        const float z = Z16 ? __half2float(__ushort_as_half(Z16[n * l.ng + g])) : 8.0f;
        gp.z = (uint32_t)(128 - (int)fminf(fmaxf(rintf(z), -100.0f), 100.0f)) * 0x01010101u;
      }
      ((GroupParam*)(ws + l.st_off))[p] = gp;
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
  __asm__ volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1"
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
  float* y;
  Layout l;
  int64_t M;
  int N;
  int row_bytes;  // of a packed weight row
  int tiles_m, tiles_n;
};

// Four waves as 2 x 2, each 32 MI rows by 32 NI weight rows.  G: group size,
// 0 for one group per row.
template <int MI, int NI, int G>
__global__ __launch_bounds__(256, 2) void w4a8_kernel(MulArgs a) {
  constexpr int TM = 64 * MI, TN = 64 * NI;
  constexpr int ABYTES = TM * KCH, BBYTES = TN * (KCH / 2), STAGE = ABYTES + BBYTES;
  constexpr int GPC = G == 0 ? 1 : KCH / G;  // groups per chunk
  __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = lane >> 5, l32 = lane & 31, wm = wave & 1, wn = wave >> 1;
  // consecutive workgroups go to the eight XCDs in turn: each XCD takes a run
  // of tiles, 8 x 8 of them at a time, so that its L2 holds what they share
  const int total = a.tiles_m * a.tiles_n, per = (total + 7) / 8;
  const int t = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (t >= min(total, ((int)(blockIdx.x & 7) + 1) * per)) return;
  const int sup = t / (8 * a.tiles_m), rest = t - sup * 8 * a.tiles_m;
  const int wn_tiles = min(8, a.tiles_n - 8 * sup);
  const int tm = rest / wn_tiles, tn = 8 * sup + rest - tm * wn_tiles;
  const int64_t m0 = (int64_t)tm * TM;
  const int n0 = tn * TN;
  const int nch = a.l.nch;

  // direct loads: X panels are copied as they are; a weight row's 64 bytes of
  // a chunk go to units that put 16 rows on different banks
  const char* xbase = a.ws + (m0 >> 5) * nch * PANEL;
  const char* qbase = (const char*)a.q + (int64_t)n0 * a.row_bytes;
  uint32_t qrow[NI], qu;
#pragma unroll
  for (int j = 0; j < NI; ++j)
    qrow[j] = (uint32_t)min(16 * (NI * wave + j) + (lane >> 2), a.N - 1 - n0) * a.row_bytes;
  qu = 16 * ((lane & 3) ^ ((lane >> 4) & 3));
  auto issue = [&](int c, int buf) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + buf * STAGE;
#pragma unroll
    for (int j = 0; j < 2 * MI; ++j) {  // 1 KB pieces of the tile's 2 MI panels
      const int piece = 2 * MI * wave + j;
      dma16(xbase + ((int64_t)(piece >> 2) * nch + c) * PANEL, (piece & 3) * 1024 + lane * 16,
            dst + piece * 1024);
    }
    const uint32_t k = min((uint32_t)c * (KCH / 2) + qu, (uint32_t)a.row_bytes - 16);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      dma16(qbase, qrow[j] + k, dst + ABYTES + (NI * wave + j) * 1024);
  };
  const GroupParam* st = (const GroupParam*)(a.ws + a.l.st_off) + n0 + 32 * NI * wn + l32;
  GroupParam gp[NI][GPC], gn[NI][GPC];
  auto params = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int g = 0; g < GPC; ++g)
        gn[j][g] = st[(int64_t)(G == 0 ? 0 : min(c * GPC + g, a.l.ng - 1)) * a.l.cols + 32 * j];
  };

  f32x16 tot[G == 0 ? 1 : MI][G == 0 ? 1 : NI];
  i32x16 sum[G == 0 ? MI : 1][G == 0 ? NI : 1];
  if constexpr (G == 0) {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[mi][ni][i] = 0;
  } else {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int i = 0; i < 16; ++i) tot[mi][ni][i] = 0.0f;
  }
  issue(0, 0);
  params(0);
  for (int c = 0; c < nch; ++c) {
    const int buf = c & 1;
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();  // chunk c has landed, and chunk c - 1's buffer is read
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int g = 0; g < GPC; ++g) gp[j][g] = gn[j][g];
    if (c + 1 < nch) {
      issue(c + 1, buf ^ 1);
      params(c + 1);
    }
    const char* la = lds + buf * STAGE + wm * MI * PANEL;
    const char* lb = lds + buf * STAGE + ABYTES + 32 * NI * wn * (KCH / 2);
    // MFMA q of a chunk takes, in lane half h, unit xu(q) of X: with groups of
    // 32 the two halves share 32 consecutive k, otherwise 64
    i32x4 bf[NI][4];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const int row = 32 * ni + l32;
      uint32_t w[8];
      if constexpr (G == 32) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint2 v = *(const uint2*)(lb + row * 64 + 16 * (q ^ ((row >> 2) & 3)) + 8 * h);
          w[2 * q] = v.x, w[2 * q + 1] = v.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 v = *(const uint4*)(lb + row * 64 + 16 * ((2 * j + h) ^ ((row >> 2) & 3)));
          w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t zc = gp[ni][q * GPC / 4].z;
        int o[4];
        minus_zero(w[2 * q], zc, o[0], o[1]);
        minus_zero(w[2 * q + 1], zc, o[2], o[3]);
        bf[ni][q] = i32x4{o[0], o[1], o[2], o[3]};
      }
    }
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      i32x4 af[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int u = G == 32 ? 2 * q + h : 4 * (q >> 1) + 2 * h + (q & 1);
        af[q] = *(const i32x4*)(la + mi * PANEL + l32 * KCH + 16 * (u ^ ((l32 >> 1) & 7)));
      }
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        if constexpr (G == 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sum[mi][ni] =
                __builtin_amdgcn_mfma_i32_32x32x32_i8(af[q], bf[ni][q], sum[mi][ni], 0, 0, 0);
        } else {
#pragma unroll
          for (int g = 0; g < GPC; ++g) {
            i32x16 acc = {};
#pragma unroll
            for (int q = 4 * g / GPC; q < 4 * (g + 1) / GPC; ++q)
              acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(af[q], bf[ni][q], acc, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              tot[mi][ni][i] = fmaf(gp[ni][g].s, (float)acc[i], tot[mi][ni][i]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t row = m0 + 32 * (MI * wm + mi) + 8 * (i >> 2) + 4 * h + (i & 3);
      if (row >= a.M) continue;
      const float sx = a.sx[row];
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        const int col = n0 + 32 * (NI * wn + ni) + l32;
        float v;
        if constexpr (G == 0)
          v = gp[ni][0].s * (float)sum[mi][ni][i];
        else
          v = tot[mi][ni][i];
        if (col < a.N) a.y[row * a.N + col] = sx * v;
      }
    }
}

struct Tile {
  int mi, ni;
};

Tile tile_for(int64_t m, int64_t d_out) {
  if (ceil_div(m, 256) * ceil_div(d_out, 128) >= 512) return {4, 2};
  if (ceil_div(m, 128) * ceil_div(d_out, 128) >= 256) return {2, 2};
  return {1, 1};
}

template <int MI, int NI>
void launch(const MulArgs& a, int G, hipStream_t stream) {
  const dim3 grid((unsigned)(8 * ceil_div((int64_t)a.tiles_m * a.tiles_n, 8)));
  switch (G) {
    case 32: hipLaunchKernelGGL((w4a8_kernel<MI, NI, 32>), grid, dim3(256), 0, stream, a); break;
    case 64: hipLaunchKernelGGL((w4a8_kernel<MI, NI, 64>), grid, dim3(256), 0, stream, a); break;
    case 128: hipLaunchKernelGGL((w4a8_kernel<MI, NI, 128>), grid, dim3(256), 0, stream, a); break;
    default: hipLaunchKernelGGL((w4a8_kernel<MI, NI, 0>), grid, dim3(256), 0, stream, a);
  }
}

}  // namespace

size_t w4a8_workspace(int64_t m, int64_t d_out, int64_t d_in, int group_size) {
  if (m <= VEC_M) return 0;
  const Tile t = tile_for(m, d_out);
  return layout_of(m, d_out, d_in, group_size, 64 * t.mi, 64 * t.ni).bytes;
}

hipError_t w4a8_launch(const int8_t* X, const float* x_scales, int64_t m, int64_t ldx,
                       const uint32_t* qweight, const uint16_t* scales_f16,
                       const uint16_t* zeros_f16, int64_t d_out, int64_t d_in, int group_size,
                       float* Y, void* ws, hipStream_t stream) {
  if (m <= VEC_M) {
    w4vec::VecArgs v;
    v.x = (const char*)X, v.sx = x_scales, v.q = qweight, v.s16 = scales_f16, v.z16 = zeros_f16;
    v.y = Y, v.ldx = ldx, v.m = (int)m, v.n = (int)d_out, v.k = (int)d_in;
    v.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
    v.vec = w4vec::scale_vec(scales_f16, zeros_f16, v.ng);
    const int G = group_size == -1 ? 0 : group_size;
    return w4vec::dot_takes(m, d_in) ? w4vec::dot_launch<true>(v, G, stream)
                                          : w4vec::vec_launch<true>(v, G, stream);
  }
  const Tile t = tile_for(m, d_out);
  const Layout l = layout_of(m, d_out, d_in, group_size, 64 * t.mi, 64 * t.ni);
  const int64_t items = l.rows * l.nch * (KCH / 16) + (int64_t)l.ng * l.cols;
  hipLaunchKernelGGL(w4a8_layout_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(items, 256), 8192)),
                     dim3(256), 0, stream, X, ldx, m, (int)d_out, (int)d_in, l, scales_f16,
                     zeros_f16, (char*)ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  MulArgs a;
  a.ws = (const char*)ws, a.sx = x_scales, a.q = qweight, a.y = Y, a.l = l, a.M = m;
  a.N = (int)d_out, a.row_bytes = (int)(d_in / 2);
  a.tiles_m = (int)(l.rows / (64 * t.mi)), a.tiles_n = (int)(l.cols / (64 * t.ni));
  const int G = group_size == -1 ? 0 : group_size;
  if (t.mi == 4)
    launch<4, 2>(a, G, stream);
  else if (t.mi == 2)
    launch<2, 2>(a, G, stream);
  else
    launch<1, 1>(a, G, stream);
  return hipGetLastError();
}

}  // namespace gptq
