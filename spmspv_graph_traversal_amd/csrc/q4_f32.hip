// The 4-bit product kernels of one x type and matrix count.
#include "q4_tiles.h"

hipError_t dbs_q4_launch_f32(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s) {
  return q4::launch<float, 1>(q, words, gpt, shape, s);
}
