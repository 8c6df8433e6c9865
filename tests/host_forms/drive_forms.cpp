// Prints the form of the 4-bit product with its epilogue that the plans choose: for each
// "m d_out d_in group gated" of the arguments a line
//   dot                                    one token by dot products
//   vec <nt> <r> <rs> <splits> <slots>     few tokens: tiles of 16 tokens and weight rows
//   tiles <wide> <splits> <least> <most>   more: blocks of 32 rows of X to a tile
#include <cstdio>
#include <cstdlib>

#include "linear_plan.h"
#include "w4_plan.h"

int main(int argc, char** argv) {
  for (int i = 1; i + 4 < argc; i += 5) {
    const int64_t m = std::atoll(argv[i]), d_out = std::atoll(argv[i + 1]), d_in = std::atoll(argv[i + 2]);
    const int g = std::atoi(argv[i + 3]);
    const bool gated = std::atoi(argv[i + 4]) != 0;
    if (gptq::linear::few_tokens(m, d_out, d_in, g)) {
      if (gptq::w4vec::dot_takes(m, d_in)) {
        std::printf("dot\n");
        continue;
      }
      const auto p = gptq::w4vec::vec_plan(false, m, d_out, d_in, g == -1 ? 0 : g, true, gated);
      std::printf("vec %d %d %d %d %d\n", (int)((m + 15) / 16), p.r, p.rs, p.splits, p.slots);
      continue;
    }
    const auto p = gptq::linear::plan_for(m, d_out, d_in, g, gated);
    const int blocks = (int)((m + 31) / 32), least = blocks / p.tiles_m;
    std::printf("tiles %d %d %d %d\n", (int)p.wide, p.splits, least, least + (blocks % p.tiles_m ? 1 : 0));
  }
}
