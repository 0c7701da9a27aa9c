// The paged cache of 4-bit keys and values (dbs_kv4_*): its layout, and what its kernels share.
#pragma once

#include "values.h"

// tokens of a block: what a wave takes of the cache at a time
#define KV4_BLOCK 32
#define KV4_MAX_DIM DBS_KV4_MAX_DIM

typedef _Float16 kv4_half2 __attribute__((ext_vector_type(2)));

// The head size that the cache holds for heads of `dim`: those that the kernels are made for.
inline int kv4_padded(int dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }

// A page's part of one key head, in bytes from its start (d: padded head size, groups: of a head):
//   key codes      [token][4 g][d/32 k] words of eight nibbles e: channel 32 k + 8 g + e
//   key records    [token][group] halves s, b
//   value codes    [token / 8][16 c][d/16 n] words of eight nibbles e: channel 16 n + c of token 8 (token / 8) + e
//   value records  [token / 8][group] eight halves s, then eight halves b, of tokens 0 4 1 5 2 6 3 7
// Keys are multiplied along their channels and values along their tokens: a word holds eight neighbours of that direction, in
// the place of the lane (g or c) that takes them, so that a lane's words are one load and an operand needs no exchange.
struct kv4_layout {
  int d, groups, key_records, value_codes, value_records, head_bytes;
  __host__ __device__ kv4_layout(int padded, int group, int page_tokens) {
    d = padded;
    groups = padded / group;
    key_records = page_tokens * padded / 2;
    value_codes = key_records + page_tokens * groups * 4;
    value_records = value_codes + page_tokens * padded / 2;
    head_bytes = value_records + page_tokens * groups * 4;
  }
};

// Waves of a SIMD that the kernel for few rows is made to hold, r tiles of 16 rows a wave, heads of 32 nc channels in groups of
// 32 gc: as many as spill no register, since a spilled one's load waits for all codes that are on their way.
constexpr int kv4_waves(int nc, int gc, int r, bool wide) {
  const int need = 8 * nc * r + 4 * nc * r * (wide ? 2 : 1) + 4 * nc + 18 * (nc / gc) + 12 * r + 35;  // output, queries, codes, records, scores
  return need <= 128 ? 4 : need <= 168 ? 3 : need <= 256 ? 2 : 1;
}

// place of token e of eight in a value record
__host__ __device__ inline int kv4_place(int e) { return (e & 3) * 2 + (e >> 2); }

// What a kernel knows of the cache and of the new tokens: sequence b's are rows [new_ptr[b], new_ptr[b + 1]), or `each` a
// sequence where new_ptr is null, the last ones of its lens[b] tokens.
struct kv4_view {
  uint8_t *pool;
  int64_t page_stride;
  int pages, page_shift, width, sequences, tokens, each;
  const int32_t *table;
  int64_t ldtable;
  const int32_t *lens, *new_ptr;
};

struct kv4_rows {
  int first, count;  // rows [first, first + count)
  int position;                // of the first one, negative where the cache holds fewer tokens than are new
};

// Tables and lists, which nothing writes while a kernel runs: read as constants, so that what all lanes read alike is a scalar load
// behind stores too.
DBS_DEV int kv4_list(const int32_t *p, int64_t at) { return ((const __attribute__((address_space(4))) int32_t *)(uintptr_t)p)[at]; }

DBS_DEV int kv4_new_ptr(const kv4_view &c, int b) { return min(max(kv4_list(c.new_ptr, b), 0), c.tokens); }

DBS_DEV kv4_rows kv4_rows_of(const kv4_view &c, int b) {
  kv4_rows r;
  r.first = c.new_ptr ? kv4_new_ptr(c, b) : b * c.each;
  r.count = c.new_ptr ? max(kv4_new_ptr(c, b + 1) - r.first, 0) : c.each;
  const int most = c.width << c.page_shift;
  r.position = min(max(kv4_list(c.lens, b), 0), most) - r.count;
  return r;
}

// The sequence that unit `u` belongs to where sequence b's units start at new_ptr[b] * times / per + extra * b: the last one
// that starts at or before u, found by a wave, 64 sequences at a time.
DBS_DEV int kv4_find(const kv4_view &c, int64_t u, int times, int per, int extra) {
  int low = 0, count = c.sequences;  // among [low, low + count)
  const int lane = threadIdx.x & 63;
  while (count > 1) {
    const int step = (count + 63) >> 6;
    const int b = low + lane * step;
    const bool at = lane * step < count && (int64_t)kv4_new_ptr(c, b) * times / per + (int64_t)extra * b <= u;
    const int last = max(63 - __clzll(__ballot(at)), 0);
    count = min(step, count - last * step);
    low += last * step;
  }
  return __builtin_amdgcn_readfirstlane(low);
}

// A page's part of a head, or null where the table names no page of the pool.
DBS_DEV uint8_t *kv4_page(const kv4_view &c, int b, int token, int64_t head_offset) {
  const int at = token >> c.page_shift;
  if (token < 0 || at >= c.width) return nullptr;
  const int page = kv4_list(c.table, b * c.ldtable + at);
  if ((unsigned)page >= (unsigned)c.pages) return nullptr;
  return c.pool + page * c.page_stride + head_offset;
}

// the attention kernels (kv4_attention.h), one file for each padded head size
struct kv4_attention_args {
  kv4_view cache;
  int device;  // the current one
  int heads_per_key, key_heads, dim, group;
  const void *q;
  int q_bf16;
  int64_t qt, qh;
  void *out;
  int out_bf16;
  int64_t ot, oh;
  float scale;  // times log2 e
  int window, sinks;
  int splits, chunk;  // blocks of a split
  float *partial;     // where splits > 1: unnormalised rows [splits][tokens][heads][d], then their bases and sums [..][2]
};

// where a split's row goes, and its base and sum
DBS_DEV float *kv4_partial(const kv4_attention_args &a, int64_t token, int head, int d) {
  const int64_t heads = (int64_t)a.key_heads * a.heads_per_key;
  return a.partial + ((blockIdx.y * (int64_t)a.cache.tokens + token) * heads + head) * d;
}
DBS_DEV void kv4_partial_end(const kv4_attention_args &a, int64_t token, int head, int d, float base, float sum) {
  const int64_t heads = (int64_t)a.key_heads * a.heads_per_key, rows = a.cache.tokens * heads;
  ((float2 *)(a.partial + a.splits * rows * d))[blockIdx.y * rows + token * heads + head] = make_float2(base, sum);
}

// tiles: 16-row tiles of a wave, 4: the kernel for many rows (kv4_prompt.h); 8: that
// with workgroups of eight waves; share: more than four waves for 16 rows; wide: q and p in two parts
hipError_t kv4_attention_64(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s);
hipError_t kv4_attention_96(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s);
hipError_t kv4_attention_128(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s);
hipError_t kv4_attention_192(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s);
hipError_t kv4_attention_256(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s);
