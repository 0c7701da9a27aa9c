// Attention over the 4-bit cache, heads of up to 64.
#include "kv4_prompt.h"

hipError_t kv4_attention_64(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s) {
  return kv4::launch<2>(a, tiles, share, wide, grid, s);
}
