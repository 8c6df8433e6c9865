// How the W4A16 product with its epilogue is laid out on the chip: which kernels, the
// form of the weights, tiles and splits.  Host code alone.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace gptq {
namespace linear {

constexpr int64_t up_to(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int KCH = 64;  // k per chunk: 128 bytes of a row of X, 32 of a weight row

// The weights in eight bits, for calls with many rows of X: q - z as e4m3, which
// has every whole number up to 16 in magnitude, so that two leave for bf16 with one
// operation and no zero is taken off again.  Panels of 32 columns x 64 k (2 KB),
// chunk after chunk, 16-byte unit u of row r at u ^ (r / 4 mod 4), as the tiles
// have them in LDS; columns past the last and k past the row's end are zeros.
// Scales follow as float32 [ng][cols].  (57344 x 8192: 0.15 ms.)
struct Wide {
  int64_t cols;  // padded to whole tiles
  int nch, ng;
  size_t scales;  // byte offset
  size_t bytes;
};

inline Wide wide_of(int64_t d_out, int64_t d_in, int group_size, bool gated) {
  Wide w;
  w.cols = up_to(gated ? up_to(d_out / 2, 32) * 64 : d_out, 256) * 256;
  w.nch = (int)up_to(d_in, KCH);
  w.ng = group_size == -1 ? 1 : (int)(d_in / group_size);
  w.scales = (size_t)w.cols * w.nch * KCH;
  w.bytes = w.scales + (size_t)w.cols * w.ng * 4;
  return w;
}

// A wave's tile: up to 256 rows of X by 32 weight rows, or, of the wide weights,
// 128 by 64.
constexpr int blocks_n(bool wide) { return wide ? 2 : 1; }
constexpr int most_m(bool wide) { return wide ? 4 : 8; }
constexpr int tile_n(bool wide) { return 128 * blocks_n(wide); }

// Few tokens: the kernels that read the weights once for all of them.  Always up to 16;
// past that their vector work grows with every 16 tokens, most with small groups, and
// past one round of workgroups nothing hides it, so large weights go to the tiles.  From
// sweeps of 19 layers of 17 to 134 million codes, gated and not (us by tiles / here):
// 24 tokens, groups of 32: 67 M 24 / 21, 71 M 26 / 28, 117 M 33 / 43; other groups up to
// 84 M a tenth to four tenths less here.  40 tokens, groups of 32: 35 M 24 / 23, 42 M
// 25 / 27, 67 M 29 / 34; of 64: 50 M 25 / 21, 59 M 26 / 28, 71 M 29 / 38; of 128: 50 M
// 24 / 19, from 59 M on the same to a tenth; one: 56 M 26 / 23, 59 M 22 / 26.  64 tokens,
// groups of 32: 17 M 21 / 21, 21 M 21 / 26; of 64: 17 M 19 / 19, 21 M 21 / 22, 26 M 22 /
// 30; of 128: 34 M 24 / 23, 42 M 25 / 24, gated 24 / 30, 59 M 27 / 31; one: 35 M 23 / 22,
// 42 M 22 / 22, gated 22 / 24, 59 M 24 / 30.
inline bool few_tokens(int64_t m, int64_t d_out, int64_t d_in, int group_size) {
  const int64_t codes = d_out * d_in;
  if (m > 64) return false;
  if (m <= 16) return true;
  if (m <= 32) return group_size != 32 || codes < 70000000;
  if (m <= 48) return group_size == 128 || codes < (group_size == 32 ? 40000000 : 55000000);
  return codes < (group_size == 32 || group_size == 64 ? 19000000 : 40000000);
}

struct Plan {
  bool wide;  // weights in eight bits first
  int tiles_m, tiles_n;
  int splits, per_split;
  size_t part_off, bytes;
};

// Tiles, splits of k and the form of the weights by the least of a time in us,
// fitted to some 300 launches of 128 to 4096 tokens through seven layers.  A chunk
// takes a tile of b blocks of 32 rows `alone` where it has a CU to itself (up to
// 256 workgroups) and `shared` where the CU has two (past 256 some have, with more
// to wait for than the mean); where the chip is full its power is the bound, and
// taking four bits apart in every tile costs a tenth more.  Making the weights wide
// costs a launch and their bytes, splits their sums' bytes.
// 515 tokens through 4099 x 11008, groups of 32: 92 us with three tiles of rows and
// k in five (98 with five and three; 106 wide); 2048 tokens through 8192 x 8192: 333
// us wide, 349 from four bits; 8192 tokens through 57344 x 8192: 7.0 and 7.6 ms.
inline Plan plan_for(int64_t m, int64_t d_out, int64_t d_in, int group_size, bool gated) {
  const int nch = (int)up_to(d_in, KCH);
  const int64_t blocks = up_to(m, 32), cols = gated ? up_to(d_out / 2, 32) * 64 : d_out;
  const bool g32 = group_size == 32;
  Plan p = {};
  double best = 0.0;
  // (a launch's threads are below 2^32)
  const bool may_widen = up_to(cols, 256) * 256 * (4 * nch) < (int64_t)1 << 31;
  for (int wide = 0; wide < 1 + may_widen; ++wide) {
    const int64_t tiles_n = up_to(cols, tile_n(wide));
    int64_t before = 0;
    for (int b = most_m(wide); b >= 1; --b) {
      const int64_t tiles_m = up_to(blocks, b);
      if (tiles_m == before) continue;  // the larger b gave the same tiles
      before = tiles_m;
      const int most = (int)up_to(blocks, tiles_m);
      const double alone = wide ? 0.26 + 0.276 * most : 0.32 + (g32 ? 0.173 : 0.146) * most;
      const double two = wide ? 0.31 + 0.511 * most : g32 ? 0.57 + 0.233 * most : 0.47 + 0.224 * most;
      for (int splits = 1; splits <= 8 && (splits == 1 || splits * 4 <= nch); ++splits) {
        const int64_t groups = tiles_m * tiles_n * splits, last = groups % 512;
        const double shared = std::max(alone, !wide && groups >= 512 ? 1.1 * two : two);
        const double end = last == 0 ? 0.0
                           : last <= 256 ? alone
                                         : alone + (shared - alone) * (0.55 + 0.45 * (double)(last - 256) / 256);
        double us = (double)up_to(nch, splits) * ((double)(groups / 512) * shared + end);
        if (splits > 1) us += 4.0e-6 * (double)(m * d_out) * (splits + 1) / 3.0;
        if (wide) us += 4.0 + 1.5e-6 * (double)(cols * d_in) / 5.0;
        if (best == 0.0 || us < best) {
          best = us;
          p.wide = wide, p.tiles_m = (int)tiles_m, p.tiles_n = (int)tiles_n, p.splits = splits;
        }
      }
    }
  }
  p.per_split = (int)up_to(nch, p.splits);
  p.splits = (int)up_to(nch, p.per_split);
  p.part_off = p.wide ? up_to(wide_of(d_out, d_in, group_size, gated).bytes, 256) * 256 : 0;
  p.bytes = p.part_off + (p.splits > 1 ? (size_t)p.splits * m * d_out * 4 : 0);
  return p;
}

}  // namespace linear
}  // namespace gptq
