// The paged cache of 4-bit keys and values: new tokens into it (dbs_kv4_store), and the calls of the attention over it
// (dbs_kv4_attention), whose kernels are in kv4_attention.h.
#include "kv4.h"

#include <math.h>

#include <type_traits>

namespace {

struct kv4_side {
  const void *x;
  int64_t xt, xh;
  void *y;
  int64_t yt, yh;
};

// another lane's value: by permutation of four lanes or from the other end of 8 or 16, an operand of the instruction that uses it
template <int HOW>
DBS_DEV float lane_swap(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), HOW, 0xF, 0xF, true));
}

/*
 * Mathematics: of a group's values x (32, 64 or 128 channels of a head of a token) b = half(min), s = half((max - b) / 15) and
 * codes rint((x - b) / s) within 0..15, each step in fp32 and with products by reciprocals, so that the codes are
 * reproducible bit by bit.  A group with a value beyond DBS_KV4_MAX_VALUE is NaN throughout.
 *
 * A workgroup takes the new ones of eight tokens that share words of the value codes, one key head after the other: lanes along
 * the channels, eight to a lane, keys in the first half of the workgroup and values in the second; the next head's are on their
 * way meanwhile.  Words of tokens that were there before are read and kept.  Only this workgroup writes these words, so nothing is
 * atomic.  Few tokens have a workgroup for each head, many share the chain of list, length and page among `per` heads (some 8000
 * tokens of 8 heads of 128 channels 24.6 us with a workgroup a head, 19.5 so).
 *
 * Bound by the launch and one chain for the tokens of a step (64 sequences 4.4 us), for prompts by the issue of vector instructions,
 * 284 of a wave for 512 values, a workgroup's beginning included: 65 MB in 18.0 us, 3.6 TB/s.
 */
template <class X, class Y>
__global__ __launch_bounds__(512) void k_kv4_store(kv4_view c, int heads, int per, int dim, int padded, int group, kv4_side key, kv4_side value) {
  __shared__ uint32_t codes[2][8][KV4_MAX_DIM / 8 + 1];
  const int64_t unit = blockIdx.x;
  int b, nth;
  if (c.new_ptr) {
    b = kv4_find(c, unit, 1, 8, 2);
    nth = (int)(unit - kv4_new_ptr(c, b) / 8 - 2 * b);
  } else {
    const int units = (c.each + 6) / 8 + 1;
    b = (int)(unit / units);
    nth = (int)(unit % units);
  }
  const kv4_rows rows = kv4_rows_of(c, b);
  if (nth < 0 || rows.count <= 0) return;
  // slots [from, from + 8) of the cache; before the first slot there is nothing to keep, but rows to return
  const int from = ((rows.position >> 3) + nth) * 8;
  if (from >= rows.position + rows.count) return;

  const int lanes = padded / 8, side = threadIdx.x >= 8 * lanes;
  const int e = threadIdx.x / lanes - 8 * side, l = threadIdx.x % lanes, channel = 8 * l;
  const int t = from + e - rows.position;  // the token among the new ones
  const bool is_new = t >= 0 && t < rows.count, in = is_new && channel < dim;
  const kv4_layout lay(padded, group, 1 << c.page_shift);
  const kv4_side &to = side ? value : key;
  const int64_t row = rows.first + t;
  const int head0 = blockIdx.y * per, head1 = min(head0 + per, heads);
  const auto load = [&](int head, X (&v)[8]) {
    if (in) __builtin_memcpy(v, (const X *)to.x + row * to.xt + head * to.xh + channel, sizeof v);
  };
  X now[8], next[8];
  load(head0, now);
  uint8_t *page = kv4_page(c, b, from, (int64_t)head0 * lay.head_bytes);
  const int slot = from & ((1 << c.page_shift) - 1);
  const bool first = channel % group == 0;
  // nibble e of a word of the value codes is token e's
  uint32_t news = 0u;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (from + k >= rows.position && from + k < rows.position + rows.count) news |= 15u << (4 * k);

  for (int head = head0; head < head1; ++head) {
    if (head + 1 < head1) load(head + 1, next);
    float x[8], low = INFINITY, high = -INFINITY;
    bool bad = false;
    if (in) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = dbs_value<X>::load(&now[i]);
        low = fminf(low, x[i]);
        high = fmaxf(high, x[i]);
        bad |= !(fabsf(x[i]) <= DBS_KV4_MAX_VALUE);
      }
    }
    if (bad) high = INFINITY;  // tells the group
    // across the 4, 8 or 16 lanes of a group, each step leaving the lanes that it joined alike
    low = fminf(low, lane_swap<0xB1>(low)), high = fmaxf(high, lane_swap<0xB1>(high));  // neighbours
    low = fminf(low, lane_swap<0x4E>(low)), high = fmaxf(high, lane_swap<0x4E>(high));  // pairs
    if (group > 32) low = fminf(low, lane_swap<0x141>(low)), high = fmaxf(high, lane_swap<0x141>(high));  // eight lanes backwards
    if (group > 64) low = fminf(low, lane_swap<0x140>(low)), high = fmaxf(high, lane_swap<0x140>(high));  // sixteen
    bad = high > DBS_KV4_MAX_VALUE;
    if (low > high) low = high = 0.0f;  // no channel of the head
    _Float16 of = (_Float16)low;
    _Float16 sc = (_Float16)fmaxf((high - (float)of) * (1.0f / 15.0f), 0.0f);
    if (bad) of = sc = (_Float16)NAN;
    const float step = (float)sc, base = (float)of, inverse = step > 0.0f ? 1.0f / step : 0.0f;
    uint32_t word = 0u;
    if (in) {
      Y y[8];
      float stands[8], codes4[2] = {};  // four codes are exact in fp32
#pragma unroll
      for (int i = 7; i >= 0; --i) {
        const float q = __builtin_amdgcn_fmed3f(rintf((x[i] - base) * inverse), 0.0f, 15.0f);
        codes4[i / 4] = __builtin_fmaf(codes4[i / 4], 16.0f, q);
        stands[i] = (float)(_Float16)__builtin_fmaf(step, q, base);
      }
      if (!bad) word = (uint32_t)codes4[0] | (uint32_t)codes4[1] << 16;
      dbs_round(y, stands);
      if (to.y) __builtin_memcpy((Y *)to.y + row * to.yt + head * to.yh + channel, y, sizeof y);
    }
    uint16_t bits[2];
    __builtin_memcpy(&bits[0], &sc, 2);
    __builtin_memcpy(&bits[1], &of, 2);
    if (page && is_new && !side) {
      // channels 32 k + 8 g .. + 7 are word g (d / 32) + k
      ((uint32_t *)(page + (slot + e) * (padded / 2)))[(l & 3) * (padded / 32) + (l >> 2)] = word;
      if (first) ((uint32_t *)(page + lay.key_records))[(slot + e) * lay.groups + channel / group] = bits[0] | (uint32_t)bits[1] << 16;
    }
    uint32_t (&words)[8][KV4_MAX_DIM / 8 + 1] = codes[(head - head0) & 1];
    if (side) {
      words[e][l] = word;
      if (page && is_new && first) {
        uint16_t *r = (uint16_t *)(page + lay.value_records) + ((slot >> 3) * lay.groups + channel / group) * 16 + kv4_place(e);
        r[0] = bits[0];
        r[8] = bits[1];
      }
    }
    __syncthreads();  // one a head: the next head's words go to the other buffer
    if (page) {
      uint32_t *out = (uint32_t *)(page + lay.value_codes) + (slot >> 3) * padded;
      for (int i = threadIdx.x; i < padded; i += blockDim.x) {
        const int ch = 16 * (i % (padded / 16)) + i / (padded / 16);
        uint32_t w = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k) w |= (words[k][ch >> 3] >> (4 * (ch & 7)) & 15u) << (4 * k);
        out[i] = news == ~0u ? w : (out[i] & ~news) | (w & news);
      }
      page += lay.head_bytes;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) now[i] = next[i];
  }
}

/*
 * Joins the splits of a row: o = sum_z 2^(m_z - m) o_z / sum_z 2^(m_z - m) l_z.  `lanes` lanes hold a row of four channels each, and
 * `parts` such groups of a workgroup take every parts-th split of it and meet in LDS, in a fixed order: all of a workgroup for one
 * row where rows are few and splits many, one group a row where rows are many.  A launch and one chain of loads, 4 us: an
 * attention of no tokens takes 7.3 us with it, 3.3 without, an empty launch 1.8.
 */
template <class Y>
__global__ __launch_bounds__(1024) void k_kv4_combine(kv4_view c, int heads, int dim, int padded, int splits, int lanes, int parts,
                                                     const float *__restrict__ partial, Y *__restrict__ out, int64_t ot, int64_t oh) {
  __shared__ float2 sums[1024];
  __shared__ float shared[1024][4];
  const int group = threadIdx.x / lanes, lane = threadIdx.x % lanes, part = group % parts;
  const int64_t all = (int64_t)c.tokens * heads, row = (int64_t)blockIdx.x * (blockDim.x / (lanes * parts)) + group / parts;
  const int64_t t = row / heads;
  const int h = (int)(row % heads);
  // a row of no sequence was written by nobody
  const bool real = row < all && !(c.new_ptr && (t < kv4_new_ptr(c, 0) || t >= kv4_new_ptr(c, c.sequences)));
  const bool in = real && 4 * lane < padded;
  const float2 *const ends = (const float2 *)(partial + splits * all * padded) + row;
  const float *const from = partial + row * padded + 4 * lane;
  float top = -3.402823466e38f, sum = 0.0f, v[4] = {};
  // Splits z0, z0 + parts, .. of a row, four on their way.  A split that saw nothing left its row as it was: `live` looks at the sums before
  // it asks for rows.
  const auto join = [&](int z0, auto live) {
    float2 e[4];
    float x[4][4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) e[k] = ends[min(z0 + k * parts, splits - 1) * all];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!decltype(live)::value || e[k].y != 0.0f) __builtin_memcpy(x[k], from + min(z0 + k * parts, splits - 1) * all * padded, 16);
    float t = top;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (z0 + k * parts >= splits) e[k] = make_float2(-3.402823466e38f, 0.0f);
      t = fmaxf(t, e[k].x);
    }
    const float f = __builtin_amdgcn_exp2f(top - t);
    top = t;
    sum *= f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float g = __builtin_amdgcn_exp2f(e[k].x - top);
      sum += g * e[k].y;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += e[k].y != 0.0f ? g * x[k][i] : 0.0f;
    }
  };
  if (in) {
    // a round trip longer, which few rows would wait for (131072 tokens 33.0 us, 34.3 with it): where lanes are left over, the first four are taken
    // unasked
    int z0 = part;
    if (parts > 1 && z0 < splits) {
      join(z0, std::false_type());
      z0 += 4 * parts;
    }
    for (; z0 < splits; z0 += 4 * parts) join(z0, std::true_type());
  }
  if (parts > 1) {
    sums[threadIdx.x] = make_float2(top, sum);
#pragma unroll
    for (int k = 0; k < 4; ++k) shared[threadIdx.x][k] = v[k];
    __syncthreads();
    if (part) return;
    float t = top;
    for (int p = 1; p < parts; ++p) t = fmaxf(t, sums[threadIdx.x + p * lanes].x);
    const float f = __builtin_amdgcn_exp2f(top - t);
    sum *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] *= f;
    for (int p = 1; p < parts; ++p) {
      const float2 e = sums[threadIdx.x + p * lanes];
      const float g = __builtin_amdgcn_exp2f(e.x - t);
      sum += g * e.y;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += g * shared[threadIdx.x + p * lanes][k];
    }
  }
  if (!in || 4 * lane >= dim) return;
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  Y y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] *= f;
  dbs_round(y, v);
  __builtin_memcpy(out + t * ot + h * oh + 4 * lane, y, sizeof y);
}

template <class Y>
hipError_t combine(const kv4_view &c, int heads, int dim, int splits, const void *partial, void *out, int64_t ot, int64_t oh, hipStream_t s) {
  const int padded = kv4_padded(dim);
  int lanes = 16, parts = 1;
  while (4 * lanes < padded) lanes *= 2;
  const int64_t rows = (int64_t)c.tokens * heads;
  // about as many lanes as the card holds at once
  while (lanes * parts < 1024 && parts < splits && rows * lanes * parts < 256 * 1024) parts *= 2;
  const int threads = lanes * parts < 256 ? 256 : lanes * parts, per = threads / (lanes * parts);
  hipLaunchKernelGGL(k_kv4_combine<Y>, dim3((unsigned)((rows + per - 1) / per)), dim3(threads), 0, s, c, heads, dim, padded, splits, lanes, parts,
                     (const float *)partial, (Y *)out, ot, oh);
  return DBS_NOTE(hipGetLastError());
}

bool view_of(const dbs_kv4_cache *a, int32_t tokens, kv4_view *c, dbs_status *st) {
  *st = DBS_ERR_INVALID_ARG;
  int64_t bytes = 0;
  if (!a || tokens < 0 || dbs_kv4_page_bytes(a->key_heads, a->head_dim, a->group, a->page_tokens, &bytes) != DBS_OK) return false;
  if (a->sequences < 0 || a->pages < 0 || a->table_pages < 0 || a->page_stride < bytes || a->page_stride % 16) return false;
  if (a->sequences > 1 && a->ldtable < a->table_pages) return false;
  if (!a->new_ptr && a->sequences > 0 && tokens % a->sequences) return false;
  if (a->sequences == 0 && tokens > 0 && !a->new_ptr) return false;
  const int64_t slots = (int64_t)a->table_pages * a->page_tokens;
  if (slots > DBS_KV4_MAX_CONTEXT || a->sequences > DBS_KV4_MAX_SEQUENCES) {
    *st = DBS_ERR_UNSUPPORTED;
    return false;
  }
  *st = DBS_OK;
  if (tokens == 0 || a->sequences == 0) return false;
  if (!a->lens || !a->pool || a->pages < 1 || (a->table_pages > 0 && !a->table) || (uintptr_t)a->pool % 16) {
    *st = DBS_ERR_INVALID_ARG;
    return false;
  }
  c->pool = (uint8_t *)a->pool;
  c->page_stride = a->page_stride;
  c->pages = a->pages;
  c->page_shift = __builtin_ctz((unsigned)a->page_tokens);
  c->width = a->table_pages;
  c->sequences = a->sequences;
  c->tokens = tokens;
  c->each = a->new_ptr ? 0 : tokens / a->sequences;
  c->table = a->table;
  c->ldtable = a->ldtable;
  c->lens = a->lens;
  c->new_ptr = a->new_ptr;
  return true;
}

// whether heads [tokens][heads][dim] share an element with each other
bool heads_meet(int64_t tokens, int64_t st, int64_t heads, int64_t sh, int64_t dim) {
  return !dbs_rows_apart(tokens, st, heads, sh, dim) && !dbs_rows_apart(heads, sh, tokens, st, dim);
}

dbs_rows rows_of(const void *p, int64_t tokens, int64_t st, int64_t heads, int64_t sh, int64_t dim, int dtype) {
  const __int128 size = dbs_vector_size(dtype);
  return {(__int128)(uintptr_t)p, tokens, st * size, heads, sh * size, dim * size};
}

bool written_over(const dbs_rows &out, const void *p, int64_t bytes) {
  const dbs_rows s = out.span();
  return p && dbs_overlap(p, bytes, (const void *)(uintptr_t)s.at, (int64_t)s.width);
}

// whether rows that a call writes meet what it reads of the cache
bool meets_lists(const dbs_rows &out, const dbs_kv4_cache *a) {
  return written_over(out, a->lens, (int64_t)a->sequences * 4) ||
         written_over(out, a->new_ptr, ((int64_t)a->sequences + 1) * 4) ||
         written_over(out, a->table, a->table_pages ? ((a->sequences - 1) * a->ldtable + a->table_pages) * 4 : 0);
}
bool meets_pool(const dbs_rows &rows, const dbs_kv4_cache *a) {
  int64_t bytes = 0;
  (void)dbs_kv4_page_bytes(a->key_heads, a->head_dim, a->group, a->page_tokens, &bytes);
  // rows between the pages of a larger buffer are no use of it: the whole span counts
  return written_over(rows, a->pool, (a->pages - 1) * a->page_stride + bytes);
}

// How a call is cut: tiles of 16 rows a wave takes (4 and 8: waves of 32 rows), workgroups along the rows, splits of the tokens, and whether
// more than four waves share 16 rows.
struct kv4_plan {
  int tiles, splits, chunk;
  bool share;
  int64_t units;
};

int64_t partial_bytes(const dbs_kv4_cache *a, int32_t tokens, int32_t heads, int splits) {
  return splits > 1 ? (int64_t)splits * tokens * heads * (kv4_padded(a->head_dim) + 2) * 4 : 0;
}

kv4_plan plan_of(const dbs_kv4_cache *a, int32_t tokens, int32_t heads, bool wide, int32_t window, int32_t sinks, int32_t max_len) {
  constexpr int units_of_card = 256;
  kv4_plan p = {};
  const int rep = heads / a->key_heads, d = kv4_padded(a->head_dim), nc = d / 32, gc = a->group / 32;
  const int64_t rows = (int64_t)tokens * rep, each = (rows + a->sequences - 1) / a->sequences;
  // Up to 64 rows two tiles a wave: 16 x 32 rows of 3000 tokens of 128 channels 24 us, 27 with one tile, 32 with the kernel for many
  // rows.  Two tiles of larger heads leave no registers; one, and many, of 256 channels 57 and 98 us, of 16 x 64 rows 101 and 96.
  p.tiles = each <= 16 ? 1 : each > 64 ? 4 : d <= 128 ? 2 : 1;
  int64_t slots = (int64_t)a->table_pages * a->page_tokens;
  if (max_len > 0 && max_len < slots) slots = max_len;
  const auto cut = [&](int per) {  // workgroups of `per` rows
    p.units = a->new_ptr ? rows / per + a->sequences : (tokens / a->sequences * (int64_t)rep + per - 1) / per * a->sequences;
  };
  const auto blocks_of = [&](int per) {  // that the rows of a workgroup see at most
    int64_t blocks = (slots + KV4_BLOCK - 1) / KV4_BLOCK;
    if (window) {
      const int64_t span = (int64_t)window + (each < per ? each : per) / rep + 1;
      const int64_t seen = (span + KV4_BLOCK - 1) / KV4_BLOCK + 1 + ((int64_t)sinks + KV4_BLOCK - 1) / KV4_BLOCK;
      if (seen < blocks) blocks = seen;
    }
    return blocks;
  };
  if (p.tiles == 4 && (d == 128 || d == 192) && !wide) {
    // Eight waves share a tile's values and are all that a compute unit holds; of workgroups of four it holds two at 128 channels, which start
    // and end sooner, and one at 192.  Eight where they fill the card, as splits of a context that is long beside the rows too; at 128
    // channels where they do so twice, tokens are many and no more rows are idle.  With 32 heads on 8, four and eight waves: of 128 channels
    // 256 rows of 8000 tokens 68 and 62 us, 4096 of 4096 188 and 169, but 2048 of 2048 63 and 73, 16 x 512 of 512 80 and 89, 16 x 96 of
    // 2000 65 and 70; of 192 channels 4096 of 4096 354 and 247, 16 x 512 of 512 170 and 133, but 1024 of 1024 49 and 62.  At 64 channels,
    // where three workgroups of four fit, 111 and 129.
    cut(256);
    const int64_t eights = p.units * a->key_heads, seen = blocks_of(256);
    const int64_t idle = a->new_ptr ? 64 : (each + 255) / 256 * 256 - (each + 127) / 128 * 128;
    const bool fill = eights >= (d == 128 ? 2 : 1) * units_of_card || (slots * rep >= 4 * each && eights * (seen / 8) >= units_of_card);
    if (fill && (d == 192 || (seen >= 48 && idle * 16 <= each))) p.tiles = 8;
  }
  const int waves = p.tiles >= 4 ? 2 : kv4_waves(nc, gc, p.tiles, wide);
  p.splits = 1;
  if (p.tiles == 1 && waves > 1) {
    // More waves, for 16 rows of a key head, where four would be split and joined by a second launch: eight of four a SIMD, so that two
    // workgroups fit, else all of a compute unit, for as many workgroups as the card holds.  With 8 key heads, four waves and more:
    // of 64 channels 16 sequences of 300 tokens 5.6 and 5.3 us, of 800 9.1 and 7.0, 60 of 500 12.4 and 8.4, one of 1500 8.7 and 9.2; of
    // 128 channels 32 of 500 11.5 and 8.8, of 1500 17.6 and 14.1, but one of 1500 9.4 and 13.1, 16 of 300 7.0 and 8.1, 60 of 500 10.6 and 16.
    cut(16);
    const int64_t groups = p.units * a->key_heads, blocks = blocks_of(16);
    const bool half = waves == 4, many = groups * 2 >= units_of_card;
    if (groups <= (half ? 2 : 1) * units_of_card && blocks >= (half && groups <= units_of_card ? 9 : 16) &&
        blocks * nc <= (!half && many ? 200 : 100)) {
      p.share = true;
      return p;
    }
  }
  const int per = p.tiles >= 4 ? 32 * p.tiles : 64 * p.tiles;
  cut(per);
  const int64_t blocks = blocks_of(per), groups = p.units * a->key_heads;
  int unit = 4;  // a split's blocks are a multiple of it
  int64_t splits = 1;
  const int64_t most = DBS_KV4_MAX_WORKSPACE / (partial_bytes(a, tokens, heads, 2) / 2);  // splits that the workspace has room for
  if (p.tiles >= 4) {
    // Splits pay where they fill the card's last round better than the joining of their rows costs: rounds of workgroups in units
    // of a block's time, 1.3 us, in which joining moves 5 MB.  The room is not what sequences have: without a bound on the workspace
    // tables of a million tokens would ask for gigabytes of it (with and without it, where the room is used: 4160 rows of 131072 tokens 8.51
    // and 8.43 ms, 8192 given by a list 15.7 and 16.0).
    const int64_t at_once = units_of_card * (p.tiles == 8 || wide || d > 128 ? 1 : 2);
    double best = 0.0;
    for (int64_t s = 1; s <= 64 && s <= most && s <= (blocks + 7) / 8; ++s) {
      const int64_t chunk = (blocks + s - 1) / s;
      const double cost = (double)((groups * s + at_once - 1) / at_once) * (chunk + 4) +
                          (s > 1 ? 4.0 + (double)s * tokens * heads * d * 8 / 5e6 : 0.0);
      if (s == 1 || cost < best) best = cost, splits = s;
    }
  } else {
    // as many workgroups as the card holds at once, of two blocks a wave at least; more of them where sequences may differ in length
    const int64_t once = units_of_card * waves, several = p.units > 1 ? 4 * once : 0;
    splits = once / groups < blocks / 8 ? once / groups : blocks / 8;
    // down to four blocks while every workgroup has a compute unit to itself, of contexts that are split at all: seven sequences of
    // 3001 tokens with 35 rows 17.5 us with eight, 15.3 so; but on shared ones seven of 1000 with 36 rows 16.2 and 20.4, and one of 300
    // with four rows 6.7 in one piece, 8.8 in two
    const int64_t fine = units_of_card / groups < blocks / 4 ? units_of_card / groups : blocks / 4;
    if (blocks >= 16 && splits < fine) splits = fine, unit = each <= 16 * p.tiles ? 4 : 2;  // by the waves that split the tokens
    const int64_t more = several / groups < blocks / 40 ? several / groups : blocks / 40;
    if (splits < more) splits = more;
    if (splits > 1024) splits = 1024;
    if (splits > most) splits = most;
  }
  if (splits < 1) splits = 1;
  p.chunk = (int)((blocks + splits - 1) / splits);
  p.chunk = (p.chunk + unit - 1) / unit * unit;
  p.splits = blocks > p.chunk ? (int)((blocks + p.chunk - 1) / p.chunk) : 1;
  return p;
}

dbs_status check_attention(const dbs_kv4_cache *a, int32_t tokens, int32_t heads, int32_t q_dtype, int32_t out_dtype, int32_t window,
                           int32_t sinks, int32_t max_len, kv4_view *c, bool *go) {
  dbs_status st;
  *go = view_of(a, tokens, c, &st);
  if (st != DBS_OK) return st;
  if (heads < 0 || heads % a->key_heads || !dbs_is_vector_dtype(q_dtype) || !dbs_is_vector_dtype(out_dtype) || window < 0 ||
      sinks < 0 || max_len < 0)
    return DBS_ERR_INVALID_ARG;
  if ((int64_t)tokens * heads > DBS_KV4_MAX_ROWS) return DBS_ERR_UNSUPPORTED;
  if (heads == 0) *go = false;
  return DBS_OK;
}

}  // namespace

extern "C" {

dbs_status dbs_kv4_page_bytes(int32_t key_heads, int32_t head_dim, int32_t group, int32_t page_tokens, int64_t *bytes) {
  if (key_heads < 1 || key_heads > 65535 || head_dim < 8 || head_dim > KV4_MAX_DIM || head_dim % 8 || !bytes) return DBS_ERR_INVALID_ARG;
  if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1))) return DBS_ERR_INVALID_ARG;
  if ((group != 32 && group != 64 && group != 128) || kv4_padded(head_dim) % group) return DBS_ERR_INVALID_ARG;
  *bytes = (int64_t)key_heads * kv4_layout(kv4_padded(head_dim), group, page_tokens).head_bytes;
  return DBS_OK;
}

dbs_status dbs_kv4_store(const dbs_kv4_cache *a, int32_t tokens, const void *k, int64_t kt, int64_t kh, const void *v, int64_t vt,
                         int64_t vh, dbs_dtype x_dtype, void *k_out, int64_t kot, int64_t koh, void *v_out, int64_t vot,
                         int64_t voh, dbs_dtype out_dtype, void *stream) {
  kv4_view c;
  dbs_status st;
  const bool go = view_of(a, tokens, &c, &st);
  if (st != DBS_OK) return st;
  if (!dbs_is_vector_dtype(x_dtype) || !dbs_is_vector_dtype(out_dtype)) return DBS_ERR_INVALID_ARG;
  if ((int64_t)tokens * a->key_heads > DBS_KV4_MAX_ROWS) return DBS_ERR_UNSUPPORTED;
  if (!go) return DBS_OK;
  if (!k || !v) return DBS_ERR_INVALID_ARG;
  const int64_t h = a->key_heads, d = a->head_dim;
  const dbs_rows in[2] = {rows_of(k, tokens, kt, h, kh, d, x_dtype), rows_of(v, tokens, vt, h, vh, d, x_dtype)};
  const dbs_rows out[2] = {rows_of(k_out, tokens, kot, h, koh, d, out_dtype), rows_of(v_out, tokens, vot, h, voh, d, out_dtype)};
  const int64_t ot[2] = {kot, vot}, oh[2] = {koh, voh}, it[2] = {kt, vt}, ih[2] = {kh, vh};
  const void *const x[2] = {k, v}, *const y[2] = {k_out, v_out};
  for (int s = 0; s < 2; ++s) {
    if (meets_pool(in[s], a)) return DBS_ERR_INVALID_ARG;
    if (!y[s]) continue;
    if (heads_meet(tokens, ot[s], h, oh[s], d) || meets_pool(out[s], a) || meets_lists(out[s], a)) return DBS_ERR_INVALID_ARG;
    const bool in_place = x[s] == y[s] && x_dtype == out_dtype && (tokens < 2 || ot[s] == it[s]) && (h < 2 || oh[s] == ih[s]);
    if (!in_place && dbs_rows_meet(in[s], out[s])) return DBS_ERR_INVALID_ARG;
    if (dbs_rows_meet(in[1 - s], out[s])) return DBS_ERR_INVALID_ARG;
  }
  if (k_out && v_out && dbs_rows_meet(out[0], out[1])) return DBS_ERR_INVALID_ARG;
  int64_t bytes = 0;
  (void)dbs_kv4_page_bytes(a->key_heads, a->head_dim, a->group, a->page_tokens, &bytes);
  const dbs_rows pool = {(__int128)(uintptr_t)a->pool, 1, 0, 1, 0, (a->pages - 1) * a->page_stride + bytes};
  if (meets_lists(pool, a)) return DBS_ERR_INVALID_ARG;
  const int padded = kv4_padded(a->head_dim);
  const int64_t units = a->new_ptr ? (int64_t)tokens / 8 + 2 * (int64_t)a->sequences + 1 : ((int64_t)c.each + 6) / 8 * a->sequences + a->sequences;
  const kv4_side ks = {k, kt, kh, k_out, kot, koh}, vs = {v, vt, vh, v_out, vot, voh};
  const auto run = x_dtype == DBS_F32 ? (out_dtype == DBS_F32 ? k_kv4_store<float, float> : k_kv4_store<float, bf16_bits>)
                                      : (out_dtype == DBS_F32 ? k_kv4_store<bf16_bits, float> : k_kv4_store<bf16_bits, bf16_bits>);
  int64_t per = units * h / 2048;  // heads of a workgroup, so that the card holds all workgroups at once
  per = per < 1 ? 1 : per > h ? h : per;
  hipLaunchKernelGGL(run, dim3((unsigned)units, (unsigned)((h + per - 1) / per)), dim3(2 * padded), 0, (hipStream_t)stream, c, (int)h, (int)per,
                     a->head_dim, padded, a->group, ks, vs);
  return DBS_NOTE(hipGetLastError()) == hipSuccess ? DBS_OK : DBS_ERR_DEVICE;
}

dbs_status dbs_kv4_attention_workspace(const dbs_kv4_cache *a, int32_t tokens, int32_t heads, dbs_dtype q_dtype, dbs_dtype out_dtype,
                                       int32_t window, int32_t sinks, int32_t max_len, int64_t *bytes) {
  if (!bytes) return DBS_ERR_INVALID_ARG;
  kv4_view c;
  bool go;
  const dbs_status st = check_attention(a, tokens, heads, q_dtype, out_dtype, window, sinks, max_len, &c, &go);
  if (st != DBS_OK) return st;
  *bytes = 0;
  if (go) {
    const kv4_plan p = plan_of(a, tokens, heads, q_dtype == DBS_F32 || out_dtype == DBS_F32, window, sinks, max_len);
    *bytes = partial_bytes(a, tokens, heads, p.splits);
  }
  return DBS_OK;
}

dbs_status dbs_kv4_attention(const dbs_kv4_cache *a, int32_t tokens, int32_t heads, const void *q, dbs_dtype q_dtype, int64_t qt,
                             int64_t qh, void *out, dbs_dtype out_dtype, int64_t ot, int64_t oh, float scale, int32_t window,
                             int32_t sinks, int32_t max_len, void *workspace, int64_t workspace_bytes, void *stream) {
  kv4_view c;
  bool go;
  const dbs_status st = check_attention(a, tokens, heads, q_dtype, out_dtype, window, sinks, max_len, &c, &go);
  if (st != DBS_OK) return st;
  const float scale2 = scale * 1.4426950408889634f;
  if (!(scale > 0.0f) || !isfinite(scale2) || workspace_bytes < 0) return DBS_ERR_INVALID_ARG;
  if (!go) return DBS_OK;
  if (!q || !out || (workspace_bytes > 0 && (!workspace || (uintptr_t)workspace % 16))) return DBS_ERR_INVALID_ARG;
  const dbs_rows in = rows_of(q, tokens, qt, heads, qh, a->head_dim, q_dtype), to = rows_of(out, tokens, ot, heads, oh, a->head_dim, out_dtype);
  if (heads_meet(tokens, ot, heads, oh, a->head_dim) || dbs_rows_meet(in, to) || meets_pool(to, a) || meets_lists(to, a))
    return DBS_ERR_INVALID_ARG;
  const bool wide = q_dtype == DBS_F32 || out_dtype == DBS_F32;
  kv4_plan p = plan_of(a, tokens, heads, wide, window, sinks, max_len);
  if (workspace_bytes < partial_bytes(a, tokens, heads, p.splits)) p.splits = 1;  // slower, and right
  if (p.splits > 1) {
    const dbs_rows scratch = {(__int128)(uintptr_t)workspace, 1, 0, 1, 0, partial_bytes(a, tokens, heads, p.splits)};
    if (written_over(in, workspace, (int64_t)scratch.width) || written_over(to, workspace, (int64_t)scratch.width) ||
        meets_pool(scratch, a) || meets_lists(scratch, a))
      return DBS_ERR_INVALID_ARG;
  }
  if (p.units * a->key_heads > 0x7FFFFF) return DBS_ERR_UNSUPPORTED;  // lanes of a launch stay within 31 bits
  int device = -1;
  if (DBS_NOTE(hipGetDevice(&device)) != hipSuccess) return DBS_ERR_DEVICE;
  kv4_attention_args k = {c, device, heads / a->key_heads, a->key_heads, a->head_dim, a->group, q, q_dtype == DBS_BF16, qt, qh, out,
                          out_dtype == DBS_BF16, ot, oh, scale2, window < DBS_KV4_MAX_CONTEXT ? window : DBS_KV4_MAX_CONTEXT,
                          sinks < DBS_KV4_MAX_CONTEXT ? sinks : DBS_KV4_MAX_CONTEXT, p.splits, p.chunk, (float *)workspace};
  const int padded = kv4_padded(a->head_dim);
  const auto run = padded == 64 ? kv4_attention_64 : padded == 96 ? kv4_attention_96 : padded == 128 ? kv4_attention_128 :
                   padded == 192 ? kv4_attention_192 : kv4_attention_256;
  const dim3 grid((unsigned)(p.units * a->key_heads), (unsigned)p.splits);
  if (run(k, p.tiles, p.share, wide, grid, (hipStream_t)stream) != hipSuccess) return DBS_ERR_DEVICE;
  if (p.splits > 1) {
    const auto join = out_dtype == DBS_F32 ? combine<float> : combine<bf16_bits>;
    if (join(c, heads, a->head_dim, p.splits, workspace, out, ot, oh, (hipStream_t)stream) != hipSuccess) return DBS_ERR_DEVICE;
  }
  return DBS_OK;
}

}  // extern "C"
