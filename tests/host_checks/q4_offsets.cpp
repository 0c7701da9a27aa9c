// Host-only check of the byte offsets that the 4-bit product kernel loads from (the library's q4.h, compiled for the host
// only; no GPU).
//
// Claim: of a column block that exists, codes and records lie within the row's descriptors; of one that does not, every 16-byte
// load starts at or behind the descriptors' end, in the 32-bit arithmetic of the kernel.
#include <stdio.h>

#include "../../spmspv_graph_traversal_amd/csrc/q4.h"

static long failures = 0, checked = 0;
#define CHECK(c, ...)          \
  do {                         \
    ++checked;                 \
    if (!(c)) {                \
      ++failures;              \
      printf("FAIL " __VA_ARGS__); \
      printf("\n");            \
    }                          \
  } while (0)

int main() {
  const int kt_max = DBS_Q4_MAX_COLUMNS / Q4_COLS;
  for (int kt : {1, 2, 7, 86, 1 << 20, kt_max}) {
    const uint64_t code_bytes = (uint64_t)kt * Q4_TILE_BYTES;
    CHECK(code_bytes < 1ull << 32, "codes kt=%d", kt);
    for (int k : {0, kt / 2, kt - 1, kt, kt + 1, kt + 48})
      for (int lane : {0, 63}) {
        const uint32_t o = q4_code_offset(k, kt, lane);
        if (k < kt) CHECK((uint64_t)o + 16 <= code_bytes && o == (uint64_t)k * Q4_TILE_BYTES + lane * 16, "code kt=%d k=%d", kt, k);
        else CHECK(o >= code_bytes && (uint64_t)o + 16 <= 1ull << 32, "no code block kt=%d k=%d: %u", kt, k, o);
      }
    for (int words : {1, 2, 4, 8}) {  // of a row in a tile
      const uint64_t rec_bytes = (uint64_t)kt * Q4_ROWS * words * 4;
      const uint32_t size = words < 4 ? words * 4 : 16;
      for (int k : {0, kt / 2, kt - 1, kt, kt + 1, kt + 48})
        for (int row : {0, 15})
          for (int i = 0; i < (words + 3) / 4; ++i) {
            const uint32_t start = q4_record_offset(k, kt, row, words), o = start + 16u * i;
            if (k < kt) CHECK((uint64_t)o + size <= rec_bytes && start == ((uint64_t)k * Q4_ROWS + row) * words * 4, "record kt=%d k=%d words=%d", kt, k, words);
            else CHECK(o >= rec_bytes && (uint64_t)o + size <= 1ull << 32, "no record kt=%d k=%d words=%d load %d: %u", kt, k, words, i, o);
          }
    }
  }
  printf("%ld checks, %ld failures\n", checked, failures);
  return failures != 0;
}
