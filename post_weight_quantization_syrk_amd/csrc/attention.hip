// Attention over packed queries and runs of keys, grouped heads:
//   out[i] = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i k_j - m_i),
// over the keys that query i sees; a query that sees none gives zeros.
//
// The query heads of a key head are rows of one tile (row = query x group +
// head), so keys and values are read once for all of them, and a single token is
// the same work with fewer rows.  Scores are formed transposed, S^T = K Q^T
// (v_mfma_f32_32x32x16_bf16): a lane then holds scores of one query only, its
// maximum and sum are in-lane but for one exchange of the two lane halves, and
// exp(S^T), rounded to bf16, is already laid out as the right operand of
// O^T = V^T P^T.  (A lane's scores are of keys 4 h .. 4 h + 3 of every eight, and
// the contraction takes keys in any order: V^T's fragments are read in that order
// by the LDS transpose read.)  Scores, maxima, sums and O stay in float32; P is
// rounded to bf16 for the matrix cores and its sum is taken over the rounded
// values, so that a row's weights add up to one; where rows are few and the matrix
// cores idle, P goes in two bf16 parts.
#include "attention_ranges.h"
#include "common.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace gptq {

namespace {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;

constexpr float NO_MAX = -3.4028235e38f;  // of a row that has seen no key yet
// O is scaled again only when a row's maximum has grown by more than 2^GROWTH
// since the last time: p is then at most 2^GROWTH, with the same relative
// rounding, and sums stay far inside float32.
constexpr float GROWTH = 8.0f;

// Unit (16 bytes) u of row r of a tile in LDS stands at u ^ swizzle(r).  A cycle
// serves 256 bytes: sixteen rows read at one unit (keys), and four rows read at
// four neighbouring units (values), fall on different banks, whatever a row's 64 DB
// bytes leave over 256.  (With three bits in place of four at DB = 4 half of the
// LDS cycles were conflicts.)
template <int DB>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (DB % 4 == 0)
    return ((r & 3) << 2) | ((r >> 2) & 3);
  else if constexpr (DB % 2 == 0)
    return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  else
    return (r >> 2) & 3;
}

// Direct global -> LDS load of 16 bytes per lane at a uniform base and a lane's
// offset: lane l's bytes land at lds_off + 16 l.  In asm, since the compiler
// would wait for every load in flight before any LDS read; the loops wait for
// them themselves.  (M0 may be used for LDS one wait state after it is written.)
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

__device__ __forceinline__ float other_half(float v) {  // of the lane 32 away
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return (threadIdx.x & 32) ? __uint_as_float(r[0]) : __uint_as_float(r[1]);
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// The sequence that a tile of rows belongs to, and its place.  Sequence s has
// its tiles from slot floor(cu[s] group / rows) + s on, which leaves room for
// them all: no prefix sum over the sequences is needed, only a search.  (Rows,
// queries times group, are below 2^31: the front end sees to that.)
struct Place {
  int64_t q0;     // first query of the sequence
  int64_t start;  // first row of its keys
  int lq, lk;     // queries and keys
  int row0, rows; // first row of the tile within the sequence; rows of the sequence
};

__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32)) << 32 |
                   __builtin_amdgcn_readfirstlane((uint32_t)v));
}

// Offsets and lengths that do not fit the arrays are brought inside them.
template <int TILE_ROWS>
__device__ __forceinline__ Place find(const AttnArgs& a, int group, int slot) {
  const int lane = threadIdx.x & 63, tq = (int)a.tq;
  int lo = 0, n = a.batch;
  while (n > 1) {
    const int step = (n + 63) / 64, at = lane * step;
    const int c = min(max(a.cu_q[lo + min(at, n - 1)], 0), tq);
    const bool le = at < n && c * group / TILE_ROWS + lo + at <= slot;
    const int i = max(__builtin_popcountll(__ballot(le)) - 1, 0);
    lo += i * step;
    n = min(step, n - i * step);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int c0 = __builtin_amdgcn_readfirstlane(a.cu_q[lo]);
  const int c1 = __builtin_amdgcn_readfirstlane(a.cu_q[lo + 1]);
  int64_t start = 0;
  int len = 0;
  if (a.kv_start) {
    start = uniform(a.kv_start[lo]);
    len = __builtin_amdgcn_readfirstlane(a.kv_len[lo]);
  }
  Place p;
  const int q0 = min(max(c0, 0), tq);
  p.q0 = q0;
  p.lq = max(min(max(c1, 0), tq) - q0, 0);
  p.rows = p.lq * group;
  p.row0 = (slot - (q0 * group / TILE_ROWS + lo)) * TILE_ROWS;
  if (!a.kv_start) start = q0, len = p.lq;
  p.start = min(max(start, (int64_t)0), a.kv_rows);
  p.lk = (int)min((int64_t)max(len, 0), a.kv_rows - p.start);
  return p;
}

// What a wave keeps of 32 rows: lane l and lane l + 32 hold row l.
template <int DB>
struct Rows {
  bf16x8 q[2 * DB];  // columns 16 i + 8 h ..
  f32x16 o[DB];      // O^T: columns 32 b + 8 (i / 4) + 4 h + i % 4
  float mc, l;       // maximum times c (log2 units); this half's sum
};

template <int DB>
__device__ __forceinline__ void no_keys(Rows<DB>& w) {
#pragma unroll
  for (int b = 0; b < DB; ++b) w.o[b] = f32x16{};
  w.mc = NO_MAX, w.l = 0.0f;
}

template <int DB>
__device__ __forceinline__ void start_rows(Rows<DB>& w, const uint16_t* qrow, int hd, int h) {
#pragma unroll
  for (int i = 0; i < 2 * DB; ++i) {
    const int d = 16 * i + 8 * h;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (d < hd) v = *(const uint4*)(qrow + d);
    __builtin_memcpy(&w.q[i], &v, 16);
  }
  // used here, so that the compiler waits for them here and not, with all direct
  // loads in flight, in every step
#pragma unroll
  for (int i = 0; i < 2 * DB; ++i) asm volatile("" : "+v"(w.q[i]));
  no_keys(w);
}

// A value's part in the products, and what is set aside where it is an infinity or a NaN:
// 1 for +inf, 128 for -inf, 16384 for a NaN, so that their sum over 16 keys, weighted by
// 1 for a key that is seen, tells which of them there were.  Whether there are any.
__device__ __forceinline__ bool set_aside(bf16x8& v, bf16x8& odd) {
  uint32_t u[4], o[4];
  __builtin_memcpy(u, &v, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = 0;
#pragma unroll
    for (int sh = 0; sh < 32; sh += 16) {
      const uint32_t e = (u[i] >> sh) & 0xffffu, is = (e & 0x7f80u) == 0x7f80u ? 0xffffu : 0u;
      const uint32_t inf = 0x3f80u + (e >> 15) * (0x4300u - 0x3f80u), code = (e & 0x7fu) ? 0x4680u : inf;
      u[i] &= ~(is << sh);
      o[i] |= (code & is) << sh;
    }
  }
  __builtin_memcpy(&v, u, 16);
  __builtin_memcpy(&odd, o, 16);
  return (o[0] | o[1] | o[2] | o[3]) != 0;
}

__device__ __forceinline__ float of_odd(float sum) {
  const float minus = floorf(sum * 0.0078125f), plus = sum - 128.0f * minus;
  const float both = (plus > 0.0f ? INFINITY : 0.0f) + (minus > 0.0f ? -INFINITY : 0.0f);
  return sum >= 16384.0f ? NAN : both;
}

// One tile of 32 KB keys, in LDS at lk and lv.  rel: the last key that the lane's
// row sees, less the tile's first; masked: some row does not see all of them.  FINE:
// the weights in two bf16 parts, a rounding of 2^-17 in place of 2^-8.  Few rows have
// it: one token's error against 64 bits 0.0018 -> 0.0016, in 11.1 us for 10.7, nothing
// where memory is the bound.  Many rows do not: with it 16384 tokens are 0.0014 off in
// place of 0.0017 (0.0014 is the rounding of the output alone) and take 6.03 ms in place
// of 4.26, seven prompts 0.00116 for 0.00133 and 176 us for 133.
//
// CAREFUL: for rows whose sums came out infinite or NaN.  A product with 0 is NaN where
// the other side is odd: a value that the row does not see (its weight is 0), a value
// that it sees (the second part of its weight may be 0, or of the other sign), a key's
// last unit in place of columns past hd (the query's are 0 there).  So those columns are
// taken as 0, and odd values apart from the others, by what the row sees of them.  (A
// prompt of 2048 tokens whose values are all NaN, 32 heads over 8: 0.50 ms, clean 0.064;
// rows gone over again key by key took 25.)
template <int DB, int KB, bool FINE, bool CAREFUL>
__device__ __forceinline__ void tile_step(Rows<DB>& w, const char* lk, const char* lv, float c,
                                          int rel, bool masked, int hd) {
  constexpr int RB = 64 * DB;
  const int lane = threadIdx.x & 63, h = lane >> 5, l32 = lane & 31;
  f32x16 s[KB];
  const int ksw = swizzle<DB>(l32);
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    s[kb] = f32x16{};
#pragma unroll
    for (int i = 0; i < 2 * DB; ++i) {
      bf16x8 k = *(const bf16x8*)(lk + (32 * kb + l32) * RB + 16 * ((2 * i + h) ^ ksw));
      if constexpr (CAREFUL) {
        if (16 * i + 8 * h >= hd) k = bf16x8{};
      }
      s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, w.q[i], s[kb], 0, 0, 0);
    }
  }
  if (masked) {
    asm volatile("");
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (32 * kb + 8 * (i >> 2) + 4 * h + (i & 3) > rel) s[kb][i] = -INFINITY;
  }
  float mx = s[0][0];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[kb][i]);
  mx = fmaxf(mx, other_half(mx)) * c;
  if (__any(mx > w.mc + GROWTH)) {
    asm volatile("");  // (stays a branch: it is hardly ever taken)
    const float mc = fmaxf(w.mc, mx), f = exp2_of(w.mc - mc);
    w.mc = mc, w.l *= f;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) w.o[b][i] *= f;
  }
  const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
  // the weights of 16 keys
  auto weights = [&](int kc, bf16x8& p, bf16x8& rest) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float e0 = exp2_of(fmaf(s[kc >> 1][8 * (kc & 1) + j], c, -w.mc));
      const float e1 = exp2_of(fmaf(s[kc >> 1][8 * (kc & 1) + j + 1], c, -w.mc));
      const bf16x2 two = {(__bf16)e0, (__bf16)e1};
      w.l = __builtin_amdgcn_fdot2_f32_bf16(two, ones, w.l, false);
      p[j] = two[0], p[j + 1] = two[1];
      if constexpr (FINE) {
        const bf16x2 left = {(__bf16)(e0 - (float)two[0]), (__bf16)(e1 - (float)two[1])};
        w.l = __builtin_amdgcn_fdot2_f32_bf16(left, ones, w.l, false);
        rest[j] = left[0], rest[j + 1] = left[1];
      }
    }
  };
  const int i16 = lane & 15, trow = 4 * h + (i16 >> 2), tu = 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
  auto values = [&](int kc, int b) __attribute__((always_inline)) {
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 16 * kc + 8 * e + trow;
      const s16x4 t = lds_read_tr16(lv + row * RB + 16 * ((4 * b + tu) ^ swizzle<DB>(row)) + 8 * (i16 & 1));
      __builtin_memcpy((char*)&v + 8 * e, &t, 8);
    }
    return v;
  };
  if constexpr (!CAREFUL) {
#pragma unroll
    for (int kc = 0; kc < 2 * KB; ++kc) {
      bf16x8 p, rest;
      weights(kc, p, rest);
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        const bf16x8 v = values(kc, b);
        w.o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p, w.o[b], 0, 0, 0);
        if constexpr (FINE) w.o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, rest, w.o[b], 0, 0, 0);
      }
    }
  } else {
#pragma unroll
    for (int kc = 0; kc < 2 * KB; ++kc) {
      bf16x8 p, rest, seen;
      weights(kc, p, rest);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = 8 * (kc & 1) + j, key = 32 * (kc >> 1) + 8 * (i >> 2) + 4 * h + (i & 3);
        // (a weight of exp(-inf) times an infinity is a NaN)
        const float one = s[kc >> 1][i] * c == -INFINITY ? 16384.0f : 1.0f;
        seen[j] = (__bf16)(key <= rel ? one : 0.0f);
      }
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        __builtin_amdgcn_sched_barrier(0);
        bf16x8 v = values(kc, b), odd;
        const bool any = set_aside(v, odd);
        w.o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p, w.o[b], 0, 0, 0);
        if constexpr (FINE) w.o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, rest, w.o[b], 0, 0, 0);
        if (__any(any)) {
          const f32x16 sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(odd, seen, f32x16{}, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 16; ++i) w.o[b][i] += of_odd(sum[i]);
        }
      }
    }
  }
}

template <int DB>
__device__ __forceinline__ bool finite(const Rows<DB>& w) {
  float t = w.l * 0.0f;
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) t = fmaf(w.o[b][i], 0.0f, t);
  return t == 0.0f;
}

struct Grid {
  int slots;     // tiles of rows, over all sequences
  int splits;    // of a tile's keys over workgroups
  float* part;   // splits > 1: O [splits][tq][hq][hd], then
  float2* stat;  // maximum and sum [tq][hq][splits]
};

// What a row's columns are multiplied with: nothing for a row that sees no key, NaN for
// one whose sum is NaN, or 0 with keys that it sees.
__device__ __forceinline__ float inverse(float l, bool sees) {
  return l > 0.0f ? 1.0f / l : sees ? NAN : l;
}

// Four columns of a row (query, head), finished or as a part.
__device__ __forceinline__ void store4(const AttnArgs& a, const Grid& g, int split, int64_t query,
                                       int head, int d, const float o[4], float mc, float l, bool sees) {
  if (d >= a.hd) return;
  if (g.splits == 1) {
    const float inv = inverse(l, sees);
    *(bf16x4*)(a.out + query * a.ldo + head * a.hso + d) =
        bf16x4{(__bf16)(o[0] * inv), (__bf16)(o[1] * inv), (__bf16)(o[2] * inv), (__bf16)(o[3] * inv)};
  } else {
    const int64_t row = query * a.hq + head;
    *(float4*)(g.part + (split * a.tq * a.hq + row) * a.hd + d) = make_float4(o[0], o[1], o[2], o[3]);
    // (a maximum of -inf: it sees keys, and weighs none)
    if (d == 0) g.stat[row * g.splits + split] = make_float2(sees && l == 0.0f ? -INFINITY : mc, l);
  }
}

// The wave's 32 rows leave: lane l's is `row` of the sequence (query, head), with l the
// whole row's sum and o its columns; sees: whether it sees a key of the wave's (the
// scores of those that it sees may all be -inf: its weights are then 0 / 0).
template <int DB>
__device__ __forceinline__ void leave(const AttnArgs& a, const Grid& g, const Place& p, bool live, int query,
                                      int head, int split, bool sees, const f32x16 (&o)[DB], float mc, float l,
                                      char* room) {
  constexpr int RB = 64 * DB;
  const int lane = threadIdx.x & 63, h = lane >> 5, l32 = lane & 31;
  if (g.splits > 1) {
    if (live) {
#pragma unroll
      for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float t[4] = {o[b][i], o[b][i + 1], o[b][i + 2], o[b][i + 3]};
          store4(a, g, split, p.q0 + query, head, 32 * b + 2 * i + 4 * h, t, mc, l, sees);
        }
    }
    return;
  }
  // by way of LDS (the wave's own 32 RB bytes), so that whole rows are stored: in
  // pieces of 8 bytes a row apart the stores took 4 us of a workgroup's time
  const float inv = inverse(l, sees);
  constexpr int SW = DB % 2 == 0 ? 7 : 3;  // units change places inside their eight, or four
  __asm__ volatile("" ::: "memory");
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *(bf16x4*)(room + l32 * RB + 16 * ((4 * b + (i >> 2)) ^ (l32 & SW)) + 8 * h) =
          bf16x4{(__bf16)(o[b][i] * inv), (__bf16)(o[b][i + 1] * inv), (__bf16)(o[b][i + 2] * inv),
                 (__bf16)(o[b][i + 3] * inv)};
  const int64_t at = live ? (p.q0 + query) * a.ldo + head * a.hso : -1;
  __asm__ volatile("" ::: "memory");  // the wave's LDS accesses keep their order
#pragma unroll
  for (int j = 0; j < 2 * DB; ++j) {
    const int i = 64 * j + lane, r = i / (4 * DB), u = (i - r * 4 * DB) ^ (r & SW);
    const uint4 v = *(const uint4*)(room + 16 * i);
    const int64_t to = __shfl(at, r);
    if (to >= 0 && 8 * u < a.hd) *(uint4*)(a.out + to + 8 * u) = v;
  }
}

// Many rows: four waves of 32 rows, which share tiles of 64 keys in LDS, two buffers
// of them; two workgroups on a CU (heads up to 128), so that one's products run while
// the other forms its weights.
//
// 16384 tokens, 64 heads of 128 over 8: 4.0 to 4.5 ms by card, 0.98 to 1.10 PF/s, where a
// library bf16 product of 8192^3 reaches 1.26 to 1.31: under it the chip's clock falls to some
// 1.6 GHz, at which the matrix cores are busy 56% of the cycles and the other vector
// instructions (maxima, exponentials, rounding: 5 to a product) 36%.  Heads of 192 7.7
// ms, 0.86 PF/s, of 256 11.9 ms, 0.74 (256 to 512 registers: one wave per SIMD), of 96
// 3.3 to 3.5 ms, 0.95, of 64 2.4 to 2.5 ms, 0.92.  Seven prompts of
// 8197 tokens in all, 32 heads: 128 to 142 us by card, 0.65 PF/s: a fifth of the
// products fall on tiles that are partly masked, starting and ending take 8 us of the
// 27 that a workgroup lives, and over the last 30 us, the first sequence's rows, half
// of the workgroups' places stand empty (all sequences' long tiles first would fill
// them, and the L2s would lose the keys that a sequence's tiles share).
//
// Tried and slower (16384 tokens, against 1.05 PF/s on the same card, unless said): the
// next tile's scores formed between this one's weights, whole tiles (0.87, spills) or
// halves (0.94; heads of 192 0.70 against 0.74 then; of 256 0.75 against 0.67, a second
// form of the loop for that width alone); eight waves in two groups that take turns
// (1.01); eight waves on 256
// rows with three buffers (1.07, but the seven prompts 161 against 144 us).  No change:
// no barrier before the rows leave, a wave's priority raised for its products, sums in
// chains.
constexpr int BM = 128, BK = 64;

// (Heads up to 64: four waves per SIMD; the careful pass alone keeps registers in memory
// for it.)
template <int DB>
__global__ __launch_bounds__(256, DB == 2 ? 4 : DB <= 4 ? 2 : 1) void attention_rows_kernel(AttnArgs a, Grid g) {
  constexpr int RB = 64 * DB, TILE = BK * RB;  // bytes of a row and of a tile
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  // key heads go to the XCDs in turn; of one sequence the later rows, which see
  // more keys, first
  const int kvh = (int)(blockIdx.x % (uint32_t)a.hk), rest = (int)(blockIdx.x / (uint32_t)a.hk);
  const int split = (int)((uint32_t)rest / (uint32_t)g.slots);
  const int slot = g.slots - 1 - (rest - split * g.slots);
  const int group = (int)((uint32_t)a.hq / (uint32_t)a.hk);
  const Place p = find<BM>(a, group, slot);
  if (p.row0 < 0 || p.row0 >= p.rows) return;
  const float c = a.scale * 1.4426950408889634f;

  // the last key that any row of the tile sees
  const int back = p.lk - p.lq;
  const int tile_last = (int)((uint32_t)min(p.row0 + BM - 1, p.rows - 1) / (uint32_t)group);
  const KeyRange keys = key_range(a.causal ? min(tile_last + back, p.lk - 1) + 1 : p.lk, BK, g.splits, split);
  const int begin = keys.begin, end = keys.end;

  // direct loads: this wave's DB KB of each tile, units past hd replaced
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  int trow[DB], tcol[DB];
#pragma unroll
  for (int j = 0; j < DB; ++j) {
    const int i = (DB * wave + j) * 64 + lane;
    trow[j] = i / (4 * DB);
    tcol[j] = 16 * min((i % (4 * DB)) ^ swizzle<DB>(trow[j]), a.hd / 8 - 1);
  }
  const char* const kb = (const char*)(a.k + p.start * a.ldk + kvh * a.hsk);
  const char* const vb = (const char*)(a.v + p.start * a.ldv + kvh * a.hsv);
  auto issue = [&](int key0, int buf) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + buf * 2 * TILE + DB * wave * 1024;
    const int most = p.lk - 1 - key0;  // rows past the last key are copies of it
    const char* const ks = kb + 2 * (int64_t)key0 * a.ldk;
    const char* const vs = vb + 2 * (int64_t)key0 * a.ldv;
#pragma unroll
    for (int j = 0; j < DB; ++j)
      dma16(ks, (uint32_t)min(trow[j], most) * (uint32_t)(2 * a.ldk) + tcol[j], dst + 1024 * j);
#pragma unroll
    for (int j = 0; j < DB; ++j)
      dma16(vs, (uint32_t)min(trow[j], most) * (uint32_t)(2 * a.ldv) + tcol[j], dst + TILE + 1024 * j);
  };
  if (begin < end) issue(begin, 0);

  // rows past the last are copies of it
  const int row0 = p.row0 + 32 * wave, row = min(row0 + l32, p.rows - 1);
  const int query = (int)((uint32_t)row / (uint32_t)group), head = kvh * group + row - query * group;
  Rows<DB> w;
  start_rows<DB>(w, a.q + (p.q0 + query) * a.ldq + head * a.hsq, a.hd, h);
  // the last key that a row sees: the lane's, the wave's first and last
  const int lim = a.causal ? min(query + back, p.lk - 1) : p.lk - 1;
  const int lim_first = __builtin_amdgcn_readlane(lim, 0), lim_last = __builtin_amdgcn_readlane(lim, 31);
  auto over_keys = [&](auto careful) __attribute__((always_inline)) {
    // (by the keys that are left: a key's number may be near 2^31)
    for (int left = end - begin, buf = 0; left > 0; left -= BK, buf ^= 1) {
      const int key0 = end - left;
      // this tile has landed, and the other buffer is read
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (left > BK) issue(key0 + BK, buf ^ 1);
      if (key0 > lim_last) continue;
      const char* const t = lds + buf * 2 * TILE;
      tile_step<DB, BK / 32, false, decltype(careful)::value>(w, t, t + TILE, c, lim - key0,
                                                              lim_first - key0 < BK - 1, a.hd);
    }
  };
  over_keys(std::false_type());
  float l = w.l + other_half(w.l);
  int* const odd = (int*)(lds + 4 * TILE);
  const bool mine = __any(!finite(w));
  if (lane == 0) odd[wave] = mine;
  __syncthreads();  // the tiles are read
  if (__builtin_expect(odd[0] | odd[1] | odd[2] | odd[3], 0)) {
    no_keys(w);
    if (begin < end) issue(begin, 0);
    over_keys(std::true_type());
    l = w.l + other_half(w.l);
    __syncthreads();
  }
  leave<DB>(a, g, p, row0 + l32 < p.rows, query, head, split, min(lim, end - 1) >= begin, w.o, w.mc, l,
            lds + wave * 32 * RB);
}

// Few rows: one tile of 32 rows, the keys in tiles of 32 that four waves (two,
// where LDS holds no more) take in turn, each with two buffers of its own, so that
// none waits for another; their sums meet at the end.  Bound by reading keys and
// values: 64 sequences of 6001 keys, 64 heads over 8: 265 us, 5.9 TB/s; of 4096 to
// 8192, 302 us, 5.3 TB/s (a large copy reaches 5.1).  One token over 4096 keys: 11.0 us
// in 20 splits, of which 2.6 are the launch of the join and 1 each the sequence's search,
// the first tile's way from memory and each of two tiles.
constexpr int FM = 32, FK = 32;
constexpr int few_waves(int DB) { return DB <= 4 ? 4 : 2; }

template <int DB>
__global__ __launch_bounds__(64 * few_waves(DB), 1) void attention_keys_kernel(AttnArgs a, Grid g) {
  constexpr int RB = 64 * DB, TILE = FK * RB, PIECES = 2 * DB, FW = few_waves(DB);
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int kvh = (int)(blockIdx.x % (uint32_t)a.hk), rest = (int)(blockIdx.x / (uint32_t)a.hk);
  const int slot = (int)((uint32_t)rest / (uint32_t)g.splits), split = rest - slot * g.splits;
  const int group = (int)((uint32_t)a.hq / (uint32_t)a.hk);
  const Place p = find<FM>(a, group, slot);
  if (p.row0 < 0 || p.row0 >= p.rows) return;
  const float c = a.scale * 1.4426950408889634f;
  const int back = p.lk - p.lq;
  const int tile_last = (int)((uint32_t)min(p.row0 + FM - 1, p.rows - 1) / (uint32_t)group);
  const KeyRange keys = key_range(a.causal ? min(tile_last + back, p.lk - 1) + 1 : p.lk, FK * FW, g.splits, split);
  const int begin = keys.begin, end = keys.end;

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds + wave * 4 * TILE;
  const char* const mine = lds + wave * 4 * TILE;
  int trow[PIECES], tcol[PIECES];
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    const int i = j * 64 + lane;
    trow[j] = i / (4 * DB);
    tcol[j] = 16 * min((i % (4 * DB)) ^ swizzle<DB>(trow[j]), a.hd / 8 - 1);
  }
  const char* const kb = (const char*)(a.k + p.start * a.ldk + kvh * a.hsk);
  const char* const vb = (const char*)(a.v + p.start * a.ldv + kvh * a.hsv);
  auto issue = [&](int key0, int buf) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + buf * 2 * TILE;
    const int most = p.lk - 1 - key0;
    const char* const ks = kb + 2 * (int64_t)key0 * a.ldk;
    const char* const vs = vb + 2 * (int64_t)key0 * a.ldv;
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
      dma16(ks, (uint32_t)min(trow[j], most) * (uint32_t)(2 * a.ldk) + tcol[j], dst + 1024 * j);
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
      dma16(vs, (uint32_t)min(trow[j], most) * (uint32_t)(2 * a.ldv) + tcol[j], dst + TILE + 1024 * j);
  };
  const int mine_left = end - begin - FK * wave;  // keys from this wave's first on
  if (mine_left > 0) issue(end - mine_left, 0);

  const int row = min(p.row0 + l32, p.rows - 1);
  const int query = (int)((uint32_t)row / (uint32_t)group), head = kvh * group + row - query * group;
  Rows<DB> w;
  start_rows<DB>(w, a.q + (p.q0 + query) * a.ldq + head * a.hsq, a.hd, h);
  const int lim = a.causal ? min(query + back, p.lk - 1) : p.lk - 1;
  const int lim_first = __builtin_amdgcn_readlane(lim, 0);
  auto over_keys = [&](auto careful) __attribute__((always_inline)) {
    for (int left = mine_left, buf = 0; left > 0; left -= FK * FW, buf ^= 1) {
      const int key0 = end - left;
      // every read of the other buffer has returned before it is written again
      __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (left > FK * FW) {
        issue(key0 + FK * FW, buf ^ 1);
        __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * PIECES) : "memory");
      } else {
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      const char* const t = mine + buf * 2 * TILE;
      tile_step<DB, FK / 32, true, decltype(careful)::value>(w, t, t + TILE, c, lim - key0,
                                                             lim_first - key0 < FK - 1, a.hd);
    }
  };
  over_keys(std::false_type());
  if (__builtin_expect(__any(!finite(w)), 0)) {
    no_keys(w);
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (the tiles are read)
    issue(end - mine_left, 0);
    over_keys(std::true_type());
  }
  const float l = w.l + other_half(w.l);
  // The waves' sums meet in LDS, where a thread takes four columns of a row: rows
  // that are not there (28 of 32 for a token of four heads) cost nothing.
  constexpr int PITCH = 32 * DB + 4;
  static_assert(FW * 256 + FW * FM * PITCH * 4 <= FW * 4 * TILE, "in the tiles' place");
  float2* const stat = (float2*)lds;                             // [FW][32]
  float* const parts = (float*)(lds + FW * 256);                 // [FW][32][PITCH]
  const int live = min(FM, p.rows - p.row0);
  __syncthreads();  // the tiles are read
  if (l32 < live) {
    if (h == 0) stat[wave * FM + l32] = make_float2(w.mc, l);
    float* const mine = parts + (wave * FM + l32) * PITCH + 4 * h;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *(float4*)(mine + 32 * b + 2 * i) = make_float4(w.o[b][i], w.o[b][i + 1], w.o[b][i + 2], w.o[b][i + 3]);
  }
  __syncthreads();
  const int per = a.hd / 4;
  for (int at = threadIdx.x; at < live * per; at += 64 * FW) {
    const int r = (int)((uint32_t)at / (uint32_t)per), d = 4 * (at - r * per);
    float mc = NO_MAX, sum = 0.0f, o[4] = {};
#pragma unroll
    for (int i = 0; i < FW; ++i) mc = fmaxf(mc, stat[i * FM + r].x);
#pragma unroll
    for (int i = 0; i < FW; ++i) {
      const float2 st = stat[i * FM + r];
      const float4 v = *(const float4*)(parts + (i * FM + r) * PITCH + d);
      const float f = exp2_of(st.x - mc);
      sum = fmaf(st.y, f, sum);
      o[0] = fmaf(v.x, f, o[0]), o[1] = fmaf(v.y, f, o[1]);
      o[2] = fmaf(v.z, f, o[2]), o[3] = fmaf(v.w, f, o[3]);
    }
    const int at_row = p.row0 + r, at_query = (int)((uint32_t)at_row / (uint32_t)group);
    const int last = a.causal ? min(at_query + back, p.lk - 1) : p.lk - 1;
    store4(a, g, split, p.q0 + at_query, kvh * group + at_row - at_query * group, d, o, mc, sum,
           min(last, end - 1) >= begin);
  }
}

// The splits' parts of a row, joined by a wave: lane s has split s's maximum and
// sum, and four columns to a lane of every `subs`-th split's O.
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, Grid g) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.tq * a.hq) return;
  const int64_t query = row / a.hq;
  const int head = (int)(row - query * a.hq);
  const int per = a.hd / 4, subs = max(64 / per, 1), sub = lane / per, d = 4 * (lane - sub * per);
  const float2 st = g.stat[row * g.splits + min(lane, g.splits - 1)];
  // rows before the first and behind the last sequence are not anyone's
  const int first = a.cu_q[0], last = a.cu_q[a.batch];
  float o[4] = {};
  float mc = lane < g.splits ? st.x : NO_MAX;
  const bool blind = __any(mc == -INFINITY);  // sees keys, whose scores are -inf
#pragma unroll
  for (int i = 1; i < 64; i *= 2) mc = fmaxf(mc, __shfl_xor(mc, i));
  const float f = lane < g.splits ? exp2_of(st.x - mc) : 0.0f;
  float l = st.y * f;
#pragma unroll
  for (int i = 1; i < 64; i *= 2) l += __shfl_xor(l, i);
  const float* p = g.part + row * a.hd + d;
  const int64_t next = a.tq * a.hq * a.hd;
  for (int s = sub; s - sub < g.splits; s += 4 * subs) {  // the same trips for every lane
    float4 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = *(const float4*)(p + min(s + i * subs, g.splits - 1) * next);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = s + i * subs;
      const float w = __shfl(f, min(at, 63));
      if (at < g.splits && sub < subs) {
        o[0] = fmaf(w, t[i].x, o[0]), o[1] = fmaf(w, t[i].y, o[1]);
        o[2] = fmaf(w, t[i].z, o[2]), o[3] = fmaf(w, t[i].w, o[3]);
      }
    }
  }
  float sum[4] = {o[0], o[1], o[2], o[3]};
  for (int i = 1; i < subs; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] += __shfl(o[k], (lane + i * per) & 63);
  if (sub != 0 || query < first || query >= last) return;
  const float inv = inverse(l, l != 0.0f || blind);
  *(bf16x4*)(a.out + query * a.ldo + head * a.hso + d) =
      bf16x4{(__bf16)(sum[0] * inv), (__bf16)(sum[1] * inv), (__bf16)(sum[2] * inv), (__bf16)(sum[3] * inv)};
}

struct Plan {
  bool few;  // rows: the kernel whose waves share the keys
  Grid g;
  size_t bytes;
};

// Few rows (up to 32 to a sequence): the kernel whose waves share the keys; its
// splits by the least of a time in us.  A workgroup is priced at 35 GB/s of keys and
// values (alone on a CU it reads 39 with heads of 64, 55 of 128, 34 of 256), all
// together at 5.4 TB/s, and 4 us besides: 16 sequences
// of 8192 keys, 8 key heads: 135 us in one piece, 105 in two, 112 in four; 24: 157
// in one, 162 in four; one sequence of 4096, one key head: 43 us in one piece, 11.2 in
// 16.  Over 221 calls of 1 to 128 sequences, 1 or 8 key heads and 256 to 16384 keys what
// it chooses takes 6% longer than the best number of splits on average (with heads of
// 128 2.5%); prices fitted to each width gave 4%.
// More rows: the same, of a tile's 64 keys at a time.  A workgroup that has a CU to
// itself takes 0.87 us for them with heads of 64, 1.09 of 128, 3.2 of 256; two on a CU
// take 1.7 times as long each (past some 128 workgroups some CUs have two; with heads
// past 128 none); starting and ending takes 6 us (and more than eight rounds of
// workgroups gain nothing); the parts go to memory and back at 6 TB/s, behind a launch
// of 4 us.  The queries' own keys count half.  256 queries of 32 heads over 4096 keys
// of 8: 77 us in one piece, 36 in eight, 48 in 16; a prompt of 512: 15 us in one, 22 in
// two; 305 queries of two heads of 256 over 857 keys: 49 us in one, 22 in six.
Plan plan_for(int64_t tq, int64_t batch, int hq, int hk, int hd, int64_t max_kv_len) {
  Plan p;
  const int group = hq / hk;
  p.few = tq * group <= batch * FM;
  const int rows = p.few ? FM : BM;
  p.g.slots = (int)(tq * group / rows + batch);
  p.g.splits = 1;
  p.g.part = nullptr, p.g.stat = nullptr;
  const int64_t tiles = std::max(batch, ceil_div(tq * group, rows)) * hk;
  if (p.few) {
    const double bytes = 4.0 * (double)max_kv_len * hd;  // of a sequence and key head
    double least = 0.0;
    for (int s = 1; s <= 32 && (s == 1 || (s * 128 <= max_kv_len && tiles * s <= 1 << 16)); ++s) {
      const int64_t n = tiles * s, full = n / 256, last = n % 256;
      double us = (double)full * 256 * (bytes / s) / 5.4e6 + 4.0 * (double)ceil_div(n, 256);
      if (last) us += std::max((double)last * (bytes / s) / 5.4e6, bytes / s / 35e3);
      if (s > 1) us += 3.0;
      if (least == 0.0 || us < least) least = us, p.g.splits = s;
    }
  } else {
    const int db = hd <= 128 ? std::max((int)ceil_div(hd, 32), 2) : hd <= 192 ? 6 : 8;
    const double step = db <= 4 ? 0.65 + 0.11 * db : 0.4 * db;  // us for 64 keys
    const int64_t there = db <= 4 ? 512 : 256;                  // workgroups at a time
    const double mean = (double)(max_kv_len - std::min(max_kv_len, tq / batch) / 2) / 64.0;
    double least = 0.0;
    for (int s = 1; s <= 32 && (s == 1 || (s * 128 <= max_kv_len && tiles * s <= 4096)); ++s) {
      const int64_t n = tiles * s;
      const double two = db <= 4 ? 1.0 + 0.7 * std::min(std::max((double)(n - 128) / 256.0, 0.0), 1.0) : 1.0;
      const double longest = (double)ceil_div(ceil_div(max_kv_len, 64), s) * step * two;
      const double all = (double)tiles * mean * step * (db <= 4 ? 1.7 : 1.0) / (double)there;
      double us = std::max(longest, all) + 6.0 * (double)ceil_div(n, there);
      if (s > 1) us += 4.0 + 2.0 * (double)s * (double)(tq * hq) * (4 * hd + 8) / 6e6;
      if (least == 0.0 || us < least) least = us, p.g.splits = s;
    }
  }
  p.bytes = p.g.splits > 1 ? (size_t)p.g.splits * tq * hq * (hd * 4 + 8) : 0;
  return p;
}

template <int DB>
hipError_t launch(const AttnArgs& a, const Plan& p, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.g.slots * a.hk * p.g.splits));
  if (p.few) {
    constexpr int FW = few_waves(DB);
    hipLaunchKernelGGL((attention_keys_kernel<DB>), grid, dim3(64 * FW), (size_t)FW * 4 * FK * 64 * DB,
                       stream, a, p.g);
  } else {
    hipLaunchKernelGGL((attention_rows_kernel<DB>), grid, dim3(256), (size_t)4 * BK * 64 * DB + 64, stream,
                       a, p.g);
  }
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace(int64_t tq, int64_t batch, int hq, int hk, int hd, int64_t max_kv_len) {
  return plan_for(tq, batch, hq, hk, hd, max_kv_len).bytes;
}

hipError_t attention_launch(const AttnArgs& a, int64_t max_kv_len, void* ws, hipStream_t stream) {
  Plan p = plan_for(a.tq, a.batch, a.hq, a.hk, a.hd, max_kv_len);
  p.g.part = (float*)ws;
  p.g.stat = (float2*)((float*)ws + (size_t)p.g.splits * a.tq * a.hq * a.hd);
  hipError_t e = a.hd <= 64    ? launch<2>(a, p, stream)
                 : a.hd <= 96  ? launch<3>(a, p, stream)
                 : a.hd <= 128 ? launch<4>(a, p, stream)
                 : a.hd <= 192 ? launch<6>(a, p, stream)
                               : launch<8>(a, p, stream);
  if (e != hipSuccess || p.g.splits == 1) return e;
  hipLaunchKernelGGL(attention_join_kernel, dim3((unsigned)ceil_div(a.tq * a.hq, 4)),
                     dim3(256), 0, stream, a, p.g);
  return hipGetLastError();
}

}  // namespace gptq
