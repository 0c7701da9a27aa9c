// The kernels that calls of 4-bit products reach (the library's own choice, compiled for the host only; no GPU).
//
//   q4_forms            for each line "bf16|f32 gated masked scale_words groups_of_a_tile rows columns tokens" of the standard
//                       input: the kernel's parameters, and whether some wave goes through a round without a column block
//   q4_forms all        the same, each line once, for counts of row blocks, column blocks and tokens up to where the choice changes no
//                       more (in steps far finer than its limits, which are factors of two apart)
#include <stdio.h>
#include <string.h>

#include <set>
#include <string>

#include "../../spmspv_graph_traversal_amd/csrc/q4_tiles.h"

// launches nothing: only the kernels' names are wanted
template <class X, int WORDS, int GPT, int MATS, int R, int TOKENS, int RW>
static std::string name(q4::form<X, WORDS, GPT, MATS, R, TOKENS, RW>, int splits, int kt) {
  splits = q4::tiling<X, MATS, R, TOKENS, RW>::fitting(splits);
  char text[96];
  snprintf(text, sizeof text, "%s words=%d gpt=%d mats=%d r=%d tokens=%d rw=%d %s", sizeof(X) == 2 ? "bf16" : "f32", WORDS, GPT, MATS, R,
           TOKENS, RW, RW > 1 && kt % splits ? "empty" : "full");
  return text;
}

static std::string form_of(bool bf16, bool gated, bool masked, int words, int gpt, int64_t m, int64_t n, int tokens) {
  const int mt = (int)((m + Q4_ROWS - 1) / Q4_ROWS), kt = (int)((n + Q4_COLS - 1) / Q4_COLS);
  const q4_shape p = q4_pick_shape(mt, kt, tokens, bf16 ? DBS_BF16 : DBS_F32, gated, masked);
  std::string at;
  auto use = [&](auto f) {
    at = name(f, p.splits, kt);
    return hipSuccess;
  };
  const hipError_t e = bf16 ? (gated ? q4::with_form<bf16_bits, 2>(words, gpt, p, use) : q4::with_form<bf16_bits, 1>(words, gpt, p, use))
                            : (gated ? q4::with_form<float, 2>(words, gpt, p, use) : q4::with_form<float, 1>(words, gpt, p, use));
  return e == hipSuccess ? at : "none";
}

int main(int argc, char **argv) {
  if (argc > 1 && !strcmp(argv[1], "all")) {
    std::set<std::string> seen;
    for (int bf16 = 0; bf16 < 2; ++bf16)
      for (int call = 0; call < 3; ++call)  // plain, gated, masked
        for (int words = 1; words <= 2; ++words)
          for (int gpt = 1; gpt <= 4; gpt *= 2)
            for (int mt = 1; mt <= 4000; mt += 1 + mt / 12)
              for (int kt = 1; kt <= 49; ++kt)
                for (int tokens : {1, 4, 5, 8, 9, 16, 17, 32, 33, 48, 49, 64, 80, 96})
                  seen.insert(form_of(bf16, call == 1, call == 2, words, gpt, (int64_t)mt * 16, (int64_t)kt * 128, tokens));
    for (const std::string &s : seen) puts(s.c_str());
    return 0;
  }
  char type[8];
  int gated, masked, words, gpt, tokens;
  long long m, n;
  while (scanf("%7s %d %d %d %d %lld %lld %d", type, &gated, &masked, &words, &gpt, &m, &n, &tokens) == 8)
    puts(form_of(!strcmp(type, "bf16"), gated, masked, words, gpt, m, n, tokens).c_str());
  return 0;
}
