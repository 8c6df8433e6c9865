// Norms of queries and keys for each head, the rotation by position, and the
// writes of keys and values to their rows (of a cache):
//   y = x w / sqrt(mean(x^2) + eps) over a head (no norm: y = x),
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin),  angle = position f_i,
// for the rot/2 pairs (a, b) of a head's first rot columns: i and i + rot/2, or
// 2i and 2i + 1.
//
// Bound by memory: each value is read once and written once.  A head's columns
// are taken as units of 8, two units per lane, such that both columns of every
// pair are in one lane: no value crosses lanes but the sum of squares.  A wave
// takes a token (a part of its heads where tokens are few) and forms the token's
// angles once, one per lane: position times frequency in float64, of which whole
// turns come off before the sine is taken in float32, so positions in the
// millions lose nothing.
#include "common.h"
#include "kernels.h"
#include "linear_epi.h"

#include <algorithm>

namespace gptq {

namespace {

constexpr int WAVES = 4;
constexpr int MAX_PAIRS = 128;

// 8 consecutive values.
template <bool F32>
__device__ __forceinline__ void load8(const char* p, float v[8]) {
  if constexpr (F32) {
    const float4 a = ((const float4*)p)[0], b = ((const float4*)p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *(const uint4*)p;
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const float v[8]) {
  bf16x8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)v[i];
  *(bf16x8*)p = o;
}

// LPH: lanes per head, a power of two.
template <int LPH, bool F32>
__global__ __launch_bounds__(64 * WAVES) void qk_norm_rope_kernel(RopeArgs a, int chunks, int per) {
  constexpr int XB = F32 ? 4 : 2, HPW = 64 / LPH;
  __shared__ float2 turns[WAVES][MAX_PAIRS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t job = (int64_t)blockIdx.x * WAVES + wave;
  const int64_t t = min(job / chunks, a.m - 1);
  const int chunk = (int)(job % chunks);
  const bool live = job < a.m * chunks;

  const int half = a.rot / 2;
  if (half) {
    const double pos = (double)a.positions[t];
    for (int i = lane; i < half; i += 64) {
      double x = pos * a.inv_freq[i] * 0.15915494309189533577;  // turns
      x -= rint(x);
      float s, c;
      sincospif((float)(2.0 * x), &s, &c);
      turns[wave][i] = make_float2(c, s);
    }
  }
  __syncthreads();
  if (!live) return;

  // units of 8 columns: lane j < pairs of units: j and j + R/2, the columns of
  // its pairs; the units that do not turn follow, two to a lane
  const int U = a.hd / 8, R = a.rot / 8, j = lane % LPH;
  const bool turning = j < R / 2;
  const int u0 = turning ? j : 2 * j, u1 = turning ? j + R / 2 : 2 * j + 1;
  const bool in0 = u0 < U, in1 = u1 < U;
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int f = a.interleaved ? (i < 4 ? 4 * u0 + i : 4 * u1 + i - 4) : 8 * j + i;
    cs[i] = turning ? turns[wave][f] : make_float2(1.0f, 0.0f);
  }
  auto weight8 = [&](const void* w, int u, bool in, float v[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = w && in ? load_as_float(w, 8 * u + i, a.w_f32) : 1.0f;
  };
  float wq0[8], wq1[8], wk0[8], wk1[8];
  weight8(a.q_weight, u0, in0, wq0);
  weight8(a.q_weight, u1, in1, wq1);
  weight8(a.k_weight, u0, in0, wk0);
  weight8(a.k_weight, u1, in1, wk1);

  int64_t kv_row = t;
  if (a.slots) kv_row = a.slots[t];
  const bool kv_in = kv_row >= 0 && kv_row < a.kv_rows;
  const int heads = a.hq + a.hk + (a.v ? a.hk : 0);
  for (int it = chunk * per; it < (chunk + 1) * per; ++it) {
    const int head = it * HPW + lane / LPH;
    const bool is_q = head < a.hq, is_v = head >= a.hq + a.hk;
    const int hh = is_q ? head : is_v ? head - a.hq - a.hk : head - a.hq;
    const bool in = head < heads && (is_q || kv_in);
    const char* src = (const char*)(is_q ? a.q : is_v ? a.v : a.k) +
                      XB * (is_q ? t * a.ldq + hh * a.hsq
                                 : is_v ? t * a.ldv + hh * a.hsv : t * a.ldk + hh * a.hsk);
    float x0[8] = {}, x1[8] = {};
    if (in && in0) load8<F32>(src + XB * 8 * u0, x0);
    if (in && in1) load8<F32>(src + XB * 8 * u1, x1);
    const bool norm = is_q ? a.q_weight != nullptr : !is_v && a.k_weight != nullptr;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
#pragma unroll
    for (int o = 1; o < LPH; o *= 2) ss += __shfl_xor(ss, o);
    if (norm) {
      const float r = 1.0f / sqrtf(ss / (float)a.hd + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x0[i] = x0[i] * r * (is_q ? wq0[i] : wk0[i]);
        x1[i] = x1[i] * r * (is_q ? wq1[i] : wk1[i]);
      }
    }
    if (turning && !is_v) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = x0[2 * i], q = x0[2 * i + 1], r = x1[2 * i], s = x1[2 * i + 1];
          x0[2 * i] = p * cs[i].x - q * cs[i].y, x0[2 * i + 1] = q * cs[i].x + p * cs[i].y;
          x1[2 * i] = r * cs[4 + i].x - s * cs[4 + i].y;
          x1[2 * i + 1] = s * cs[4 + i].x + r * cs[4 + i].y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = x0[i], q = x1[i];
          x0[i] = p * cs[i].x - q * cs[i].y, x1[i] = q * cs[i].x + p * cs[i].y;
        }
      }
    }
    uint16_t* dst = is_q ? a.q_out + t * a.ldqo + hh * a.hsqo
                    : is_v ? a.v_out + kv_row * a.ldvo + hh * a.hsvo
                           : a.k_out + kv_row * a.ldko + hh * a.hsko;
    if (in && in0) store8(dst + 8 * u0, x0);
    if (in && in1) store8(dst + 8 * u1, x1);
  }
}

template <int LPH>
void launch(const RopeArgs& a, bool f32, hipStream_t stream) {
  const int heads = a.hq + a.hk + (a.v ? a.hk : 0), iters = (int)ceil_div(heads, 64 / LPH);
  // a wave per token where these fill the chip, else a token's heads over several
  const int want = (int)std::min<int64_t>(iters, ceil_div(8192, a.m));
  const int per = (int)ceil_div(iters, want), chunks = (int)ceil_div(iters, per);
  const dim3 grid((unsigned)ceil_div(a.m * chunks, WAVES));
  if (f32)
    hipLaunchKernelGGL((qk_norm_rope_kernel<LPH, true>), grid, dim3(64 * WAVES), 0, stream, a, chunks, per);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<LPH, false>), grid, dim3(64 * WAVES), 0, stream, a, chunks, per);
}

}  // namespace

hipError_t qk_norm_rope_launch(const RopeArgs& a, bool f32, hipStream_t stream) {
  // lanes that the units take, two to a lane
  const int lanes = (a.hd / 8 + 1) / 2;
  if (lanes <= 4)
    launch<4>(a, f32, stream);
  else if (lanes <= 8)
    launch<8>(a, f32, stream);
  else
    launch<16>(a, f32, stream);
  return hipGetLastError();
}

}  // namespace gptq
