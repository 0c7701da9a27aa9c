// Attention over the 4-bit cache, heads of up to 128.
#include "kv4_prompt.h"

hipError_t kv4_attention_128(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s) {
  return kv4::launch<4>(a, tiles, share, wide, grid, s);
}
