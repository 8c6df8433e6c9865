// Norms of queries and keys for each head, the rotation by position, and the
// writes of keys and values to their rows (of a cache):
//   y = x w / sqrt(mean(x^2) + eps) over a head (no norm: y = x),
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin),  angle = position f_i,
// for the rot/2 pairs (a, b) of a head's first rot columns: i and i + rot/2, or
// 2i and 2i + 1.
//
// Bound by memory: each value is read once and written once.  16384 tokens of 64 + 8
// + 8 heads of 128, bf16, take 128 us, 5.2 TB/s (a large copy reaches 5.1); 4096
// tokens of 48 heads 23.7 us, 4.3 TB/s (19.7 where the last-level cache has the inputs);
// one token 3.9 us, a launch and its loads.
// A head's columns are taken as units of 8, two units per lane, such that both
// columns of every pair are in one lane: no value crosses lanes but the sum of
// squares.  A wave takes a token, or a part of its heads, with the next heads' loads
// in flight, and forms the token's angles once, one per lane: position times
// frequency in float64, of which whole turns come off before the sine is taken in
// float32, so positions in the millions lose nothing.  Waves in flight count for
// more than loads per wave: two steps' loads ahead took 161 us, with cosines and
// weights in registers 142; they are read from LDS for every head.
#include "common.h"
#include "kernels.h"
#include "linear_epi.h"

#include <algorithm>
#include <type_traits>

namespace gptq {

namespace {

constexpr int WAVES = 4;
constexpr int MAX_PAIRS = 128;

// A unit, 8 consecutive values, as it is in memory.
template <bool F32>
struct Unit {
  uint4 u[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ void widen(const Unit<F32>& r, float v[8]) {
  if constexpr (F32) {
    __builtin_memcpy(v, r.u, 32);
  } else {
    const uint32_t u[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
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

// Sum over the LPH (4, 8 or 16) lanes of a head, in each of them: swaps inside
// fours, then mirrors of eight and sixteen.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
  auto add = [&](auto ctrl) __attribute__((always_inline)) {
    v += __int_as_float(
        __builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  add(std::integral_constant<int, 0xB1>());   // quad_perm 1 0 3 2
  add(std::integral_constant<int, 0x4E>());   // quad_perm 2 3 0 1
  if constexpr (LPH >= 8) add(std::integral_constant<int, 0x141>());   // row_half_mirror
  if constexpr (LPH >= 16) add(std::integral_constant<int, 0x140>());  // row_mirror
  return v;
}

// LPH: lanes per head, a power of two.
template <int LPH, bool F32>
__global__ __launch_bounds__(64 * WAVES, F32 ? 5 : 6) void qk_norm_rope_kernel(RopeArgs a, int chunks, int per) {
  constexpr int XB = F32 ? 4 : 2, HPW = 64 / LPH;
  __shared__ float2 turns[WAVES][MAX_PAIRS];
  __shared__ __attribute__((aligned(16))) float weights[2][8 * 2 * LPH];  // of queries and keys
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t job = (int64_t)blockIdx.x * WAVES + wave;
  const int64_t t = min(job / chunks, a.m - 1);
  const int chunk = (int)(job % chunks), first = chunk * per;
  const bool live = job < a.m * chunks;

  // units of 8 columns: lane j < pairs of units: j and j + R/2, the columns of
  // its pairs; the units that do not turn follow, two to a lane
  const int U = a.hd / 8, R = a.rot / 8, j = lane % LPH;
  const bool turning = j < R / 2;
  const int u0 = turning ? j : 2 * j, u1 = turning ? j + R / 2 : 2 * j + 1;
  const bool in0 = u0 < U, in1 = u1 < U;
  const int heads = a.hq + a.hk + (a.v ? a.hk : 0);

  // the heads of step `it` as they are in memory, one step ahead
  Unit<F32> r0 = {}, r1 = {};
  auto fetch = [&](int it) __attribute__((always_inline)) {
    const int head = it * HPW + lane / LPH;
    if (head >= heads) return;
    const bool is_q = head < a.hq, is_v = head >= a.hq + a.hk;
    const int hh = is_q ? head : is_v ? head - a.hq - a.hk : head - a.hq;
    const char* src = (const char*)(is_q ? a.q : is_v ? a.v : a.k) +
                      XB * (t * (is_q ? a.ldq : is_v ? a.ldv : a.ldk) +
                            hh * (is_q ? a.hsq : is_v ? a.hsv : a.hsk));
    if (in0) __builtin_memcpy(&r0, __builtin_assume_aligned(src + XB * 8 * u0, 16), 8 * XB);
    if (in1) __builtin_memcpy(&r1, __builtin_assume_aligned(src + XB * 8 * u1, 16), 8 * XB);
  };
  fetch(first);
  int64_t kv_row = t;
  if (a.slots) kv_row = a.slots[t];

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
  for (int i = threadIdx.x; i < 2 * a.hd; i += 64 * WAVES) {
    const int k = i >= a.hd, d = i - k * a.hd;
    const void* w = k ? a.k_weight : a.q_weight;
    weights[k][d] = w ? load_as_float(w, d, a.w_f32) : 1.0f;
  }
  __syncthreads();
  if (!live) return;

  // (cosines, sines and weights are read again for every head: the registers that
  // would hold them are worth more as waves)
  const float2* const cs0 = turns[wave] + (turning ? a.interleaved ? 4 * u0 : 8 * j : 0);
  const float2* const cs1 = turns[wave] + (turning ? a.interleaved ? 4 * u1 : 8 * j + 4 : 0);
  const bool kv_in = kv_row >= 0 && kv_row < a.kv_rows;
  for (int it = first; it < first + per; ++it) {
    const int head = it * HPW + lane / LPH;
    const bool is_q = head < a.hq, is_v = head >= a.hq + a.hk;
    const int hh = is_q ? head : is_v ? head - a.hq - a.hk : head - a.hq;
    const bool in = head < heads && (is_q || kv_in);
    float x0[8], x1[8];
    widen<F32>(r0, x0);
    widen<F32>(r1, x1);
    if (it + 1 < first + per) fetch(it + 1);
    const bool norm = is_q ? a.q_weight != nullptr : !is_v && a.k_weight != nullptr;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
    ss = head_sum<LPH>(ss);
    float eps = (float)a.eps;
    // squares past float32's end, or below its normal numbers where eps does not hide
    // that: the head times a power of two, eps times its square (an infinity stays one)
    const float up = ss / (float)a.hd + eps < 0x1p-90f ? 0x1p100f : ss > 3.4028235e38f ? 0x1p-70f : 1.0f;
    if (__builtin_expect(__any(norm && up != 1.0f), 0)) {
      const float k = norm ? up : 1.0f;
      ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x0[i] *= k, x1[i] *= k;
        ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
      }
      ss = head_sum<LPH>(ss);
      eps = (float)(a.eps * k * k);
    }
    if (norm) {
      const float r = 1.0f / sqrtf(ss / (float)a.hd + eps);
      const float* w = weights[is_q ? 0 : 1];
      // (units that are not there: their values are 0)
      const float* const w0 = w + 8 * min(u0, U - 1);
      const float* const w1 = w + 8 * min(u1, U - 1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x0[i] = x0[i] * r * w0[i];
        x1[i] = x1[i] * r * w1[i];
      }
    }
    if (turning && !is_v) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c0 = cs0[i], c1 = cs1[i];
          const float p = x0[2 * i], q = x0[2 * i + 1], r = x1[2 * i], s = x1[2 * i + 1];
          x0[2 * i] = p * c0.x - q * c0.y, x0[2 * i + 1] = q * c0.x + p * c0.y;
          x1[2 * i] = r * c1.x - s * c1.y, x1[2 * i + 1] = s * c1.x + r * c1.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 c = i < 4 ? cs0[i] : cs1[i - 4];
          const float p = x0[i], q = x1[i];
          x0[i] = p * c.x - q * c.y, x1[i] = q * c.x + p * c.y;
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
  // five steps of heads to a wave at most, or as few as fill the chip with waves
  // (16384 tokens of 80 heads, ten steps: 128 us in five and five, 140 in one run of
  // ten, 150 in single steps, whose waves each form the token's angles)
  const int want = (int)std::min<int64_t>(iters, std::max(ceil_div(iters, 5), ceil_div(8192, a.m)));
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
