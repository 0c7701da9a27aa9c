// Layout of a matrix of 4-bit codes with group scales (dbs_q4_build).
#pragma once

#include "values.h"

// Tiles of 16 rows x 128 columns in row-block order, 1 KB of codes each: 16
// bytes for each lane of a wave, in lane order.  Lane l holds row l & 15; its
// dword s (0..3) holds the eight codes of columns 32 s + 8 (l >> 4) + e, which
// is the operand a 16x16x32 matrix instruction takes from that lane in step s.
// Within the dword the code of column e starts at bit (4 n + 3) mod 32 with
// n = e / 2 + 4 (e % 2), so that after a right rotation by 4 p the codes of
// columns 2p and 2p + 1 stand in bits 3..6 and 19..22, the upper mantissa bits
// of two bf16.  A tile past the matrix's edge is filled with zero weights.
#define Q4_ROWS 16
#define Q4_COLS 128
#define Q4_TILE_BYTES 1024

// Beside each tile one record per row and group, [row][group of the tile]:
// the scale and the offset 16 + zero point of the codes read as bf16 16..31.
// bf16 scales: one word, scale << 16 | offset as bf16 (exact); fp32 scales: two
// fp32 words.
__host__ __device__ inline int q4_record_words(dbs_dtype scale_dtype) { return scale_dtype == DBS_F32 ? 2 : 1; }

// Byte offsets in a row of tiles that a lane's 16 bytes of codes and its row's records start at: column block k, if it comes
// before `end`, else one from which every load of 16 bytes is out of range of the row's descriptor, with no 32-bit sum that
// wraps: the last 16 bytes of the range, or, for records of eight words, which take two loads, some before.  (0xFFFFFFF0 fits
// in an instruction, another value takes a register: one more than the 80 that leave room for six waves in the kernel of one
// token and many rows.)
__host__ __device__ inline uint32_t q4_no_block(int words) { return words > 4 ? 0xFFFFFF00u : 0xFFFFFFF0u; }
__host__ __device__ inline uint32_t q4_code_offset(int k, int end, int lane) {
  return k < end ? (uint32_t)k * Q4_TILE_BYTES + lane * 16 : q4_no_block(4);
}
__host__ __device__ inline uint32_t q4_record_offset(int k, int end, int row, int words) {
  return k < end ? ((uint32_t)k * Q4_ROWS + row) * (words * 4) : q4_no_block(words);
}

__host__ __device__ inline int q4_code_bit(int e) { return (4 * (e / 2 + 4 * (e & 1)) + 3) & 31; }

struct dbs_q4_matrix {
  int device;
  int32_t m, n, group;
  dbs_dtype scale_dtype;
  int32_t mt, kt;   // row blocks of 16, column blocks of 128
  int32_t gpt;      // groups of a tile: 128 / group
  uint32_t *codes;  // [mt][kt][64][4]
  uint32_t *recs;   // [mt][kt][16][gpt][words]
  int64_t bytes;
};

// code of column e in a lane's dword
DBS_DEV uint32_t q4_code(uint32_t w, int e) {
  const int b = q4_code_bit(e);
  return __funnelshift_r(w, w, b) & 15u;
}

template <int WORDS>
DBS_DEV void q4_record(const uint32_t *recs, int64_t i, float &scale, float &off) {
  if (WORDS == 1) {
    const uint32_t w = recs[i];
    scale = __uint_as_float(w & 0xFFFF0000u);
    off = __uint_as_float(w << 16);
  } else {
    scale = __uint_as_float(recs[2 * i]);
    off = __uint_as_float(recs[2 * i + 1]);
  }
}
