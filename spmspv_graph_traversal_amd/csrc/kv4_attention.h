// Attention over the cache of 4-bit keys and values (kv4.h) on the matrix cores.
#pragma once

#include <type_traits>

#include "kv4.h"

namespace kv4 {

typedef kv4_half2 half2_t;
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLow = -3.402823466e38f;  // a maximum before any score
// Exponentials are 2^(score - base), the base being 10 below the largest score when it was last raised, which is when one is 15 above it: up to
// 2^15, the largest being 2^10 or more.  Halves lose bits of those below 2^-14 and end at 2^-24: a weight of one half is off by 2^-11 of itself
// or 2^-35 of the largest, one of two by 2^-23 or 2^-35.
constexpr float kBelow = 10.0f, kMost = 15.0f;
constexpr float kFar = 0x1p23f;  // a base from which on fp32 has steps of 1 and more

// The base for a largest score, at least the one before.  Where fp32 has steps of 16, 10 below is 16 below.
DBS_DEV float raised(float most, float top) {
  const float below = most - kBelow;
  return fmaxf(most - below > kMost ? most : below, top);
}

DBS_DEV half2_t as_half2(uint32_t w) { return __builtin_bit_cast(half2_t, w); }
DBS_DEV uint32_t as_bits(half2_t h) { return __builtin_bit_cast(uint32_t, h); }

// constants in registers: from literals the compiler makes two instructions of an "and or"
struct code_masks {
  uint32_t low, high, base;
  DBS_DEV code_masks() : low(0x000F000Fu), high(0x00F000F0u), base(0x64006400u) { asm("" : "+s"(low), "+s"(high), "+v"(base)); }
};

// The eight codes of a word as s q + b, in pairs of nibbles (0, 4), (1, 5), (2, 6), (3, 7): four bits under the exponent of
// 1024 are 1024 + q or 1024 + 16 q, exactly, then q, and one rounding of s q + b, which is the definition.  Thirteen
// instructions.
DBS_DEV half8_t values_of(uint32_t w, const code_masks &m, const half2_t (&s)[4], const half2_t (&b)[4]) {
  const uint32_t v = w >> 8;
  const half2_t lowered = {(_Float16)-1024.0f, (_Float16)-1024.0f}, sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f},
                lowered16 = {(_Float16)-64.0f, (_Float16)-64.0f};
  half2_t r[4];
  r[0] = as_half2((w & m.low) | m.base) + lowered;
  r[1] = __builtin_elementwise_fma(as_half2((w & m.high) | m.base), sixteenth, lowered16);
  r[2] = as_half2((v & m.low) | m.base) + lowered;
  r[3] = __builtin_elementwise_fma(as_half2((v & m.high) | m.base), sixteenth, lowered16);
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_elementwise_fma(r[i], s[i], b[i]);
  half8_t o;
  __builtin_memcpy(&o, r, 16);
  return o;
}
DBS_DEV half8_t values_of(uint32_t w, const code_masks &m, uint32_t record) {
  const half2_t sb = as_half2(record), s = {sb.x, sb.x}, b = {sb.y, sb.y};
  const half2_t ss[4] = {s, s, s, s}, bb[4] = {b, b, b, b};
  return values_of(w, m, ss, bb);
}

// sum + h.x + h.y in fp32.  Sums are of the halves that weigh the values, so that their rounding is no error of a row's total; a
// block's or tile's apart before they join the total, beside which a small one alone would lose its bits.
DBS_DEV float sum_of(half2_t h, float sum) { return __builtin_amdgcn_fdot2(h, half2_t{(_Float16)1.0f, (_Float16)1.0f}, sum, false); }

// Two halves of which either is infinite or NaN.
DBS_DEV bool not_finite(uint32_t pair) { return (pair & 0x7C00u) == 0x7C00u || (pair & 0x7C000000u) == 0x7C000000u; }

// What a pair of records makes of code 15: finite if and only if scale, offset and the values of all codes are.
DBS_DEV half2_t last_value(uint32_t s, uint32_t b) {
  return __builtin_elementwise_fma(as_half2(s), half2_t{(_Float16)15.0f, (_Float16)15.0f}, as_half2(b));
}
// x + 0 v: NaN from the first v that is not finite on
DBS_DEV half2_t or_nan(half2_t x, half2_t v) { return __builtin_elementwise_fma(v, half2_t{}, x); }
DBS_DEV bool is_nan(half2_t x) { return x.x != x.x || x.y != x.y; }

/*
 * A lane's part of a query on its way: N runs of eight channels from `first` on, `step` apart.  All loads are issued together, from
 * addresses that are there (a run behind the head is the last one again), and nothing is waited for until halves() makes halves of
 * them in the order of values_of, scaled by a power of two so that the row's largest element is between 2^14 and 2^15;
 * the lanes of a row are `lanes` apart.
 */
template <int N, bool WIDE>
struct query {
  uint4 raw[N][2];
  DBS_DEV void load(const kv4_attention_args &a, int64_t token, int head, int first, int step) {
    if (a.q_bf16) {
      const bf16_bits *const p = (const bf16_bits *)a.q + token * a.qt + head * a.qh;
#pragma unroll
      for (int n = 0; n < N; ++n) __builtin_memcpy(&raw[n][0], p + min(first + n * step, a.dim - 8), 16);
    } else {
      const float *const p = (const float *)a.q + token * a.qt + head * a.qh;
#pragma unroll
      for (int n = 0; n < N; ++n) __builtin_memcpy(raw[n], p + min(first + n * step, a.dim - 8), 32);
    }
  }
  // The scores' scale.  A product's sum is below 2^39 (256 channels of 2^15 by 2^16), and two that differ do so by 2^-48 or more.  With a
  // scale of 2^87 scores stay within fp32 and the largest has all the weight, as with any larger scale; with one of 2^-126 all are
  // nothing beside 1, as with any smaller one, but minus infinity times it is not NaN.
  template <int LANES>
  DBS_DEV float halves(const kv4_attention_args &a, bool real, int first, int step, half8_t (&high)[N], half8_t (&low)[N]) {
    float x[N][8], most = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const bool in = real && first + n * step < a.dim;
      uint32_t w[8];
      __builtin_memcpy(w, raw[n], 32);
      if (a.q_bf16) {
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          const uint32_t two = w[e];
          w[2 * e] = two << 16;
          w[2 * e + 1] = two & 0xFFFF0000u;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[n][e] = in ? __uint_as_float(w[e]) : 0.0f;
        most = fmaxf(most, fabsf(x[n][e]));
      }
    }
    for (int o = LANES; o < 64; o <<= 1) most = fmaxf(most, __shfl_xor(most, o));
    const int up = most > 0.0f && most < INFINITY ? 14 - ilogbf(most) : 0;
    if (most == INFINITY) x[0][0] = NAN;  // scores that are all minus infinity have no softmax, and would be those of a row that sees nothing
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = ldexpf(x[n][e / 2 + e % 2 * 4], up);
        high[n][e] = (_Float16)v;
        if (WIDE) low[n][e] = (_Float16)(v - (float)high[n][e]);
      }
    return __builtin_amdgcn_fmed3f(ldexpf(a.scale, -up), 0x1p-126f, 0x1p87f);
  }
};

// Words of codes, which a step reads once: past the caches, where the next layers' codes push them out anyway (131072 tokens 35.5 ->
// 33.6 us, 64 sequences of 374 MB 83.7 -> 80.9; 32 MB that the Infinity Cache would have kept 13.1 -> 13.3).
template <int N>
DBS_DEV void read_codes(uint32_t (&to)[N], const uint8_t *from) {
  constexpr int n = N % 4 ? N % 2 ? 1 : 2 : 4;
  typedef uint32_t words __attribute__((ext_vector_type(n)));
#pragma unroll
  for (int i = 0; i < N / n; ++i) {
    const words w = __builtin_nontemporal_load((const words *)from + i);
    __builtin_memcpy(to + n * i, &w, sizeof w);
  }
}

// A block of 32 tokens as a lane holds it.
template <int NC, int NG>
struct block {
  uint32_t k[2][NC], kr[2][NG], v[2 * NC], vr[NG][8];
};

/*
 * Mathematics: o_i = sum_j e_ij v_j / sum_j e_ij, e_ij = 2^(scale q_i k_j - m_i), over blocks of 32 tokens with a running
 * base m_i.  A row is one query head of one token; the rows of a key head (its query heads of all new tokens of a
 * sequence) read the same keys and values, so they fill the tiles of the matrix instructions together.
 *
 * A block's scores are K Q^T, two products of 16 tokens by 16 rows, and its output V^T P^T.  Tokens are dealt to the score
 * tiles so that the lane which gets the scores of a row's tokens 8 g .. 8 g + 7 is the one that gives them to the second
 * product: no exchange, no LDS.  Codes become halves in registers (values_of), as exact as the cache's definition.
 *
 * The base is raised, and the output scaled, only where a score is 12 above it, so that most blocks need no exchange
 * between lanes.  Sums of exponentials stay in each lane until the end.
 *
 * A workgroup's four waves split rows first (R tiles of 16 each) and, where the rows do not need them all, the tokens; further
 * splits of the tokens over workgroups are joined by k_kv4_combine.  16 rows over few tokens are one workgroup's of W waves, more than four,
 * which all split the tokens.
 *
 * What bounds it: memory where contexts are long, the launch and one chain of length, page, codes, two products and a reduction
 * where they are short.  With 32 heads of 128 channels on 8: one token of 131072 33.3 us, 143 MB at 4.3 TB/s; 64 sequences of
 * 2000 to 8000 tokens 81 us, 374 MB at 4.6 TB/s (a large copy reaches 4.7); one token of 1500 9.4 us, of none 7.3 with the joining launch
 * and 3.3 without.  In fp32, twice the products and conversions: 131072 tokens 41 us, the 64 sequences 91.
 */
template <int NC, int GC, int R, bool WIDE>
struct wave_state {
  static constexpr int NG = NC / GC, NV = 2 * NC, PARTS = WIDE ? 2 : 1, D = 32 * NC;
  half8_t q[PARTS][R][NC];
  float scale[R], top[R], sum[R];
  int position[R];  // of the lane's row, -1 behind the last
  f32x4 o[R][NV];

  DBS_DEV void scores(const block<NC, NG> &b, const code_masks &m, f32x4 (&s)[2][R]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < R; ++r) s[t][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const half8_t k = values_of(b.k[t][c], m, b.kr[t][c / GC]);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int p = 0; p < PARTS; ++p) s[t][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[p][r][c], s[t][r], 0, 0, 0);
      }
    }
  }

  // Scores become exponentials.
  DBS_DEV void soften(f32x4 (&s)[2][R]) {
#pragma clang fp contract(off)  // one rounding of a score, for the base as for its exponential: no power passes 2^kMost, however large scores are
    bool raise = false;
    float most[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float a = s[0][r][0];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) a = fmaxf(a, s[t][r][e]);
      most[r] = a * scale[r];
      raise |= most[r] - top[r] > kMost;  // exact where they are near; a sum would round
    }
    if (__builtin_expect(__any(raise), 0)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float a = raised(most[r], top[r]);
        a = fmaxf(a, __shfl_xor(a, 16));
        a = fmaxf(a, __shfl_xor(a, 32));
        const float f = __builtin_amdgcn_exp2f(top[r] - a);
        top[r] = a;
        sum[r] *= f;
#pragma unroll
        for (int n = 0; n < NV; ++n) o[r][n] *= f;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][r][e] = __builtin_amdgcn_exp2f(s[t][r][e] * scale[r] - top[r]);
  }

  DBS_DEV void weigh(const block<NC, NG> &b, const code_masks &m, const f32x4 (&s)[2][R]) {
    half8_t p[PARTS][R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      half2_t h[4], l[4];
      float of = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = half2_t{(_Float16)s[0][r][e], (_Float16)s[1][r][e]};
        of = sum_of(h[e], of);
        if (WIDE) {
          l[e] = half2_t{(_Float16)(s[0][r][e] - (float)h[e].x), (_Float16)(s[1][r][e] - (float)h[e].y)};
          of = sum_of(l[e], of);
        }
      }
      sum[r] += of;
      __builtin_memcpy(&p[0][r], h, 16);
      if (WIDE) __builtin_memcpy(&p[PARTS - 1][r], l, 16);
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      half2_t vs[4], vb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        vs[e] = as_half2(b.vr[n / (2 * GC)][e]);
        vb[e] = as_half2(b.vr[n / (2 * GC)][4 + e]);
      }
      const half8_t v = values_of(b.v[n], m, vs, vb);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < PARTS; ++i) o[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[i][r], o[r][n], 0, 0, 0);
    }
  }
};

template <int NC, int GC, int R, bool WIDE, int W>
__global__ __launch_bounds__(64 * W, kv4_waves(NC, GC, R, WIDE)) void k_kv4_attention(kv4_attention_args a) {
  typedef wave_state<NC, GC, R, WIDE> state;
  constexpr int NG = state::NG, NV = state::NV, D = state::D, ROWS = W > 4 ? 16 * R : 64 * R;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int i = lane & 15, g = lane >> 4;
  const kv4_view &c = a.cache;
  const int rep = a.heads_per_key, head = blockIdx.x % a.key_heads;
  const int64_t unit = blockIdx.x / a.key_heads;

  // the workgroup's rows
  int b, tile;
  if (c.new_ptr) {
    b = kv4_find(c, unit, rep, ROWS, 1);
    tile = (int)(unit - (int64_t)kv4_new_ptr(c, b) * rep / ROWS - b);
  } else {
    const int tiles = (int)(((int64_t)c.each * rep + ROWS - 1) / ROWS);
    b = (int)(unit / tiles);
    tile = tiles - 1 - (int)(unit % tiles);  // the longest ones first
  }
  const kv4_rows rows = kv4_rows_of(c, b);
  const int all_rows = rows.count * rep, row0 = tile * ROWS;  // DBS_KV4_MAX_ROWS keeps them within 31 bits
  if (tile < 0 || row0 >= all_rows) return;  // rows before the first sequence, or a unit with none
  const int have = min(all_rows - row0, ROWS);
  const int row_waves = have <= 16 * R ? 1 : have <= 32 * R ? 2 : 4;
  const int token_waves = W / row_waves, part = wave % token_waves;
  const int wave_row = row0 + wave / token_waves * (16 * R);  // may be behind the last row

  // What depends on no length is asked for first: the queries and, without a window, the pages of the first block.
  state w;
  query<NC, WIDE> q[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = wave_row + 16 * r + i;
    const bool real = row < all_rows;
    const int t = (real ? row : 0) / rep;
    w.position[r] = real ? rows.position + t : -1;
    q[r].load(a, rows.first + t, head * rep + (real ? row : 0) - t * rep, 8 * g, 32);
  }
  const int32_t *const table = c.table + b * c.ldtable;
  const int block0 = (a.splits > 1 ? blockIdx.y * a.chunk : 0) + part, token0 = min(block0, 1 << 25) * KV4_BLOCK;
  int early[2] = {-1, -1};
  if (c.width > 0)
#pragma unroll
    for (int h = 0; h < 2; ++h) early[h] = kv4_list(table, min((token0 + 16 * h) >> c.page_shift, c.width - 1));

  // the tokens that the wave's rows see: those below `end` from `start` on, and of the first ones `sink_blocks` blocks
  const int first_token = wave_row / rep, last_token = (min(all_rows, wave_row + 16 * R) - 1) / rep;
  const int low = rows.position + first_token, high = rows.position + last_token;  // positions of the first and last row
  const int end = wave_row < all_rows ? max(high + 1, 0) : 0;
  int start = 0, sink_blocks = 0;
  if (a.window) {
    start = max(low - a.window + 1, 0) & ~(KV4_BLOCK - 1);
    sink_blocks = (min(a.sinks, end) + KV4_BLOCK - 1) / KV4_BLOCK;
    if (sink_blocks * KV4_BLOCK >= start) start = sink_blocks = 0;
  }
  const int blocks = sink_blocks + (end > start ? (end - start + KV4_BLOCK - 1) / KV4_BLOCK : 0);
  int next = block0, stop = blocks;
  if (a.splits > 1 && blockIdx.y + 1 < a.splits) stop = min((int)(blockIdx.y + 1) * a.chunk, blocks);

  const kv4_layout lay(D, 32 * GC, 1 << c.page_shift);
  const int64_t head_offset = (int64_t)head * lay.head_bytes;
  const code_masks masks;
  const int page_mask = (1 << c.page_shift) - 1;

  auto token_of = [&](int n) { return n < sink_blocks ? n * KV4_BLOCK : start + (n - sink_blocks) * KV4_BLOCK; };
  // the pages of the block's two halves of 16 tokens, -1 where there is none
  struct place {
    int token, page[2];
  };
  auto find = [&](int n) {  // n < stop: the table has entries
    place p;
    p.token = token_of(n);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int page = kv4_list(table, min((p.token + 16 * h) >> c.page_shift, c.width - 1));
      p.page[h] = p.token + 16 * h < end && (unsigned)page < (unsigned)c.pages ? page : -1;
    }
    return p;
  };
  // A half without a page reads the pool's first, and nobody sees what it read.  Codes of keys and of values have as many bytes a
  // token, and so have their records: two bases and a lane's constants reach all four.  Where pages have 32 tokens and more both
  // halves are of one page, and the bases are the same for all lanes.
  const bool one_page = c.page_shift >= 5;
  const int k_half = i >> 3, v_half = g >> 1, k_row = 8 * ((i >> 2) & 1) + (i & 3), v_row = 8 * (g & 1);
  const int k_from = k_row + (one_page ? 16 * k_half : 0), v_from = v_row + (one_page ? 16 * v_half : 0);  // tokens from the base
  const uint32_t k_codes = k_from * (D / 2) + g * (4 * NC), k_records = lay.key_records + k_from * (4 * NG);
  const uint32_t v_codes = lay.value_codes + v_from * (D / 2) + i * (8 * NC), v_records = lay.value_records + v_from * (4 * NG);
  struct bases {
    const uint8_t *codes, *records;
  };
  auto bases_of = [&](const place &p, int h) {
    const uint8_t *const page = c.pool + (int64_t)max(p.page[h], 0) * c.page_stride + head_offset;
    const int row = (p.token + 16 * h) & page_mask;
    return bases{page + row * (D / 2), page + row * (4 * NG)};
  };
  auto lane_bases = [&](const place &p, int half) {
    const bases lo = bases_of(p, 0), hi = bases_of(p, 1);
    return bases{half ? hi.codes : lo.codes, half ? hi.records : lo.records};
  };
  auto get_keys = [&](const bases &p, block<NC, NG> &x) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      read_codes(x.k[t], p.codes + k_codes + t * (2 * D));
      __builtin_memcpy(x.kr[t], __builtin_assume_aligned(p.records + k_records + t * (16 * NG), NG % 4 ? NG % 2 ? 4 : 8 : 16), 4 * NG);
    }
  };
  auto get_values = [&](const bases &p, block<NC, NG> &x) {
    read_codes(x.v, p.codes + v_codes);
    __builtin_memcpy(x.vr, __builtin_assume_aligned(p.records + v_records, 16), 32 * NG);
  };
  auto load_keys = [&](const place &p, block<NC, NG> &x) {
    if (one_page) get_keys(bases_of(p, 0), x);
    else get_keys(lane_bases(p, k_half), x);
  };
  auto load_values = [&](const place &p, block<NC, NG> &x) {
    if (one_page) get_values(bases_of(p, 0), x);
    else get_values(lane_bases(p, v_half), x);
  };

  // A block: its scores, its weights, its values; the next one's codes on their way as registers fall free.
  block<NC, NG> x;
  place p, ahead;
  auto attend = [&] {
    f32x4 s[2][R];
    w.scores(x, masks, s);
    load_keys(ahead, x);
    const int j = p.token;
    // bit t: a row at `position` sees token j + t, one whose window begins with that of a row at `from`
    auto seen = [&](int position, int from) {
      uint32_t see = position < j ? 0u : position - j >= 31 ? ~0u : (2u << (position - j)) - 1u;
      if (a.window) {
        const int begin = from - a.window + 1 - j, sinks = a.sinks - j;
        uint32_t in = begin <= 0 ? ~0u : begin >= 32 ? 0u : ~((1u << begin) - 1u);
        in |= sinks <= 0 ? 0u : sinks >= 32 ? ~0u : (1u << sinks) - 1u;
        see &= in;
      }
      if (p.page[0] < 0) see &= 0xFFFF0000u;
      if (p.page[1] < 0) see &= 0x0000FFFFu;
      return see;
    };
    const bool whole = p.page[0] >= 0 && p.page[1] >= 0 && j + KV4_BLOCK - 1 <= low &&
                       (!a.window || j > high - a.window || j + KV4_BLOCK <= a.sinks);
    uint32_t bad[NG], some = 0u;  // the same in all lanes
    if (!whole) {
      half2_t wrong = {};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t see = seen(w.position[r], w.position[r]) >> (8 * g);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(see >> (4 * t + e) & 1u)) s[t][r][e] = -INFINITY;
      }
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) wrong = or_nan(wrong, last_value(x.vr[n][e], x.vr[n][4 + e]));
      // Nothing times a value that is not finite would be NaN: values that no row sees become 0, and one that is not finite and
      // that some rows see is added to those alone.
      if (__builtin_expect(__any(is_nan(wrong)), 0)) {
        const uint32_t any = seen(high, low);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          uint32_t mask = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t &sc = x.vr[n][e], &of = x.vr[n][4 + e];
              const uint32_t bit = 1u << (8 * g + e + 4 * h), half = h ? 0xFFFF0000u : 0x0000FFFFu;
              if (!not_finite(as_bits(last_value(sc, of)) & half)) continue;
              mask |= any & bit;
              sc &= ~half;
              of &= ~half;
            }
          mask |= (uint32_t)__shfl_xor((int)mask, 16);
          mask |= (uint32_t)__shfl_xor((int)mask, 32);
          bad[n] = (uint32_t)__builtin_amdgcn_readfirstlane((int)mask);
          some |= bad[n];
        }
      }
    }
    w.soften(s);
    w.weigh(x, masks, s);
    load_values(ahead, x);
    if (__builtin_expect(some != 0u, 0)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t see = seen(w.position[r], w.position[r]);
#pragma unroll
        for (int n = 0; n < NV; ++n)
          if (bad[n / (2 * GC)] & see) w.o[r][n] += NAN;
      }
    }
  };

  auto prepare = [&] {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w.scale[r] = q[r].template halves<16>(a, w.position[r] >= 0, 8 * g, 32, w.q[0][r], w.q[state::PARTS - 1][r]);
      w.top[r] = kLow;
      w.sum[r] = 0.0f;
#pragma unroll
      for (int n = 0; n < NV; ++n) w.o[r][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  };
  if (next < stop) {
    if (a.window) {
      p = find(next);
    } else {
      p.token = token0;
#pragma unroll
      for (int h = 0; h < 2; ++h) p.page[h] = token0 + 16 * h < end && (unsigned)early[h] < (unsigned)c.pages ? early[h] : -1;
    }
    load_keys(p, x);
    load_values(p, x);
    // Pages one block further ahead than codes.  Behind the last block it is asked for again: a branch there would have every wait be
    // for all codes that may be on their way, and a copy of the block for the last one would not fit the instruction cache as well.
    ahead = find(min(next + token_waves, stop - 1));
    prepare();
    for (; next < stop; next += token_waves) {
      attend();
      p = ahead;
      ahead = find(min(next + 2 * token_waves, stop - 1));
    }
  } else {
    prepare();
  }

  // sums over the lanes of a row; then the waves that split its tokens
#pragma unroll
  for (int r = 0; r < R; ++r) {
    w.sum[r] += __shfl_xor(w.sum[r], 16);
    w.sum[r] += __shfl_xor(w.sum[r], 32);
  }
  // four channels of a row, from 16 n + 4 g on
  auto write = [&](int r, int n, const f32x4 &o, float sum) {
    const int row = wave_row + 16 * r + i;
    if (row >= all_rows) return;
    const int64_t at_token = rows.first + row / rep;
    const int at_head = head * rep + row % rep, channel = 16 * n + 4 * g;
    if (a.splits > 1) {
      if (sum != 0.0f) __builtin_memcpy(kv4_partial(a, at_token, at_head, D) + channel, &o, 16);
      return;
    }
    if (channel >= a.dim) return;
    // a row that sees nothing is 0; a sum that is not a number stays one
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float v[4] = {o[0] * f, o[1] * f, o[2] * f, o[3] * f};
    if (a.out_bf16) {
      bf16_bits y[4];
      dbs_round(y, v);
      __builtin_memcpy((bf16_bits *)a.out + at_token * a.ot + at_head * a.oh + channel, y, 8);
    } else {
      __builtin_memcpy((float *)a.out + at_token * a.ot + at_head * a.oh + channel, v, 16);
    }
  };
  auto write_end = [&](int r, float top, float sum) {
    const int row = wave_row + 16 * r + i;
    if (a.splits > 1 && row < all_rows && g == 0) kv4_partial_end(a, rows.first + row / rep, head * rep + row % rep, D, top, sum);
  };
  if (token_waves == 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int n = 0; n < NV; ++n) write(r, n, w.o[r][n], w.sum[r]);
      write_end(r, w.top[r], w.sum[r]);
    }
    return;
  }
  // the waves that split a row's tokens put theirs into LDS, and join and write a share of the channels each
  constexpr int HALF = W <= 4 ? NV < 8 ? NV : 8 : 4;
  __shared__ f32x4 shared[W][HALF][64];
  __shared__ float2 ends[W][64];
  const int first = wave - part;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int half = 0; half < NV; half += HALF) {
      if (r + half) __syncthreads();
#pragma unroll
      for (int n = 0; n < HALF; ++n)
        if (half + n < NV) shared[wave][n][lane] = w.o[r][half + n];
      ends[wave][lane] = make_float2(w.top[r], w.sum[r]);
      __syncthreads();
      float top = kLow, sum = 0.0f, f[W];
#pragma unroll
      for (int k = 0; k < W; ++k) top = fmaxf(top, ends[k < token_waves ? first + k : wave][lane].x);
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const float2 e = ends[k < token_waves ? first + k : wave][lane];
        f[k] = k < token_waves ? __builtin_amdgcn_exp2f(e.x - top) : 0.0f;
        if (k < token_waves) sum += f[k] * e.y;
      }
      for (int n = part; n < HALF && half + n < NV; n += token_waves) {
        f32x4 o = f[0] * shared[first][n][lane];
#pragma unroll
        for (int k = 1; k < W; ++k)
          if (k < token_waves) o += f[k] * shared[first + k][n][lane];
        write(r, half + n, o, sum);
      }
      if (half == 0 && part == 0) write_end(r, top, sum);
    }
}

template <int NC, int GC, int R, bool WIDE, int W = 4>
hipError_t launch(const kv4_attention_args &a, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((k_kv4_attention<NC, GC, R, WIDE, W>), grid, dim3(64 * W), 0, s, a);
  return DBS_NOTE(hipGetLastError());
}

}  // namespace kv4
