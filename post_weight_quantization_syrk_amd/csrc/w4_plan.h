// How the products of packed 4-bit weights with a few tokens are laid out on the chip:
// weight rows to a workgroup, waves, splits.  Host code alone.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace gptq {
namespace w4vec {

constexpr int64_t up_to(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int KCH = 128;   // k per step
constexpr int KBLK = 512;  // k per block: whole scale runs for every group size

constexpr int RUN = 2048;  // k of a wave that takes one token

// One token, and a row of X that 16 waves hold.  (For two to four tokens the
// registers of X leave too few waves: the kernel for a few tokens is faster.)
constexpr bool dot_takes(int64_t m, int64_t k) { return m == 1 && k <= 16 * RUN; }

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

// Waves share the tokens' buffers only where these are large: bf16, past 32
// tokens (17 to 32: 32 tokens through 28672 x 8192 take 51 us either way).
constexpr int SHARE = 4;
constexpr bool may_share(bool i8, int nt) { return !i8 && nt >= 3; }

struct VecPlan {
  int r;   // tiles of 16 weight rows per wave
  int rs;  // waves that share the tokens' buffers
  int splits, per_split;
  int slots;
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
// With an epilogue (`finished`; gated, row tiles come in pairs and r is even) joining
// splits costs more, and up to 16 tokens of layers past one round of workgroups take
// 32 rows and four k slots each, so that several share a CU and one loads while
// another multiplies: 16 tokens through 22016 x 4096, groups of 64: 17.8 us, with 64
// rows and eight slots 21; 8 tokens 16.2 and 18.9; 57344 x 8192 64 and 71 us (12288 x
// 4096, one round of 48 rows and eight slots: 8.2 us, in 32 and four 11.1).
inline VecPlan vec_plan(bool i8, int64_t m, int64_t n, int64_t k, int G, bool finished = false,
                        bool gated = false) {
  VecPlan p = {gated ? 2 : 1, 1, 1, 1, 8, 0};
  const int nt = (int)up_to(m, 16), nblk = (int)up_to(k, KBLK);
  double least = 0.0;
  for (int rs = 1; rs <= SHARE; rs += SHARE - 1)
    for (int r = rs == 1 ? 1 : 2; r <= 4; ++r)
      for (int s = 1; s <= 8 && s <= nblk; ++s) {
        if (rs > 1 && !may_share(i8, nt)) continue;
        if (gated && r % 2 != 0) continue;
        const int per = (int)up_to(nblk, s), waves = std::min(per, most_slots(i8, nt, r, G, rs));
        const int64_t groups = up_to(n, 16 * r * rs) * s;
        const bool several = 2 * group_bytes(i8, nt, r, G, rs, waves) <= LDS_BYTES;  // per CU
        const double rounds =
            several ? std::max(1.0, groups / 256.0) : (double)up_to(groups, 256);
        const double steps = 2.0 * (up_to(per, waves) + (double)per / waves);  // most and mean
        double us = rounds * 0.27 * (2 + r) * (1.0 + 0.35 * (nt - 1)) * steps;
        if (rs > 1) us = 6.0 + us * (G == 32 ? 1.4 : G == 64 ? 1.25 : 1.0);
        if (!several) us += 2.0 * (rounds - 1.0);  // a round's start and end
        if (s > 1) us += (finished ? 6.5 : 2.5) + 1e-6 * (double)(m * n) * (s + 1);
        if (least == 0.0 || us < least) {
          least = us;
          p.r = r, p.rs = rs, p.per_split = per, p.splits = (int)up_to(nblk, per);
        }
        if (per <= waves) break;  // a wave has one block: no fewer steps
      }
  if (finished && nt == 1 && n > 12288)
    p.r = 2, p.rs = 1, p.splits = 1, p.per_split = nblk, p.slots = 4;
  p.ws_bytes = p.splits > 1 ? (size_t)p.splits * m * n * 4 : 0;
  return p;
}

}  // namespace w4vec
}  // namespace gptq
