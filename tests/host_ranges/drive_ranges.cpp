// Prints what attention_ranges.h gives: for each "kend step splits" argument triple a
// line of that triple and its runs, begin:end.
#include <cstdio>
#include <cstdlib>

#include "attention_ranges.h"

int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    const int kend = std::atoi(argv[i]), step = std::atoi(argv[i + 1]), splits = std::atoi(argv[i + 2]);
    std::printf("%d %d %d", kend, step, splits);
    for (int s = 0; s < splits; ++s) {
      const gptq::KeyRange r = gptq::key_range(kend, step, splits, s);
      std::printf(" %d:%d", r.begin, r.end);
    }
    std::printf("\n");
  }
}
