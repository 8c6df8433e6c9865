// The keys that each workgroup of a tile of rows goes over, for host and device.
#pragma once

#include <cstdint>

namespace gptq {

struct KeyRange {
  int begin, end;
};

// Keys 0 .. kend - 1 (kend <= 0: none) in `splits` runs of whole tiles of `step`: run
// `split`.  kend may be any int: in 32 bits without sign, where the last run's end in
// whole tiles, below kend + (splits + 1) step, still fits.
constexpr KeyRange key_range(int kend, int step, int splits, int split) {
  const uint32_t keys = kend > 0 ? (uint32_t)kend : 0u, s = (uint32_t)step, n = (uint32_t)splits;
  const uint32_t tiles = (keys + s - 1) / s, per = (tiles + n - 1) / n * s;
  const uint32_t begin = (uint32_t)split * per, end = begin + per;
  return {(int)(begin < keys ? begin : keys), (int)(end < keys ? end : keys)};
}

}  // namespace gptq
