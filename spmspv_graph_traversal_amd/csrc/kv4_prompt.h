// Attention of many rows over the cache of 4-bit keys and values.
#pragma once

#include <atomic>

#include "kv4_attention.h"

namespace kv4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// kinds of instructions, to __builtin_amdgcn_sched_group_barrier
constexpr int kSchedVector = 0x2, kSchedMatrix = 0x8, kSchedRead = 0x100;

/*
 * The mathematics of k_kv4_attention for the rows of a prompt, where the matrix cores and the exponentials bound it and not
 * the cache.  A workgroup takes 32 rows a wave and goes through the tokens in tiles.  It turns the codes of a tile into halves
 * once for all its waves, in LDS, in the order in which the products take them: 16 bytes a lane, so that neither writes nor reads
 * meet in a bank.  The codes of the next tile are on their way meanwhile, in registers, and there are two tiles in LDS, so that a
 * tile costs one barrier.
 *
 * What bounds it: a product takes 16 cycles of a SIMD's issue and 32 of its matrix unit, another vector instruction 4 (an
 * exponential 8).  Of 64 tokens of 128 channels a wave issues 32 products (512 cycles, 1024 of the matrix unit) and, of eight waves, 260
 * others (1180): 1690 cycles, and takes about 2400, since waves wait for each other's pipe and at the barrier.  One sequence of
 * 8192 tokens with 32 heads of 128 channels on 8 takes 607 to 632 us, 870 to 906 TFLOP/s (a large bf16 product reaches 1185 here).
 * Operands read four products ahead and exponentials dealt among the products are 2 to 6 % of it.  Slower: the next tile's values
 * between the score products (708 us, 649 then), halves of the waves in opposite order (628, 604 then).  The next tile's scores between
 * this one's exponentials spill, and wave priorities change nothing.
 *
 * Products are 32 x 32 x 16: scores K Q^T of 32 tokens by 32 rows, outputs V^T P^T of 32 channels by 32 rows.  Row m of a key
 * operand is token (m with bits 2 and 3 exchanged), so that the lane which gets a row's scores of tokens 16 u + 8 h .. + 7 is the
 * one that gives them to the second product.
 */
template <int NC, int GC, bool WIDE, int W>
struct prompt {
  static constexpr int NG = NC / GC, D = 32 * NC, PARTS = WIDE ? 2 : 1;
  static constexpr int TOKENS = NC <= 6 || !WIDE ? 64 : 32,  // as registers allow; 64 against 32 at 192 channels 571 and 747 us
                       SB = TOKENS / 32, CUT = W * 16 / TOKENS, KW = NC / CUT;  // words a thread takes of K and of V
  static constexpr int ROWS = 32 * W;
  static_assert(NC % CUT == 0, "whole words");
  static constexpr int kOperands = SB * 2 * NC * 64;  // of K or of V
  static constexpr int kFlags = NG * (TOKENS / 8);    // bytes
  static constexpr size_t kLds = 2 * (2 * kOperands * 16 + (kFlags + 15) / 16 * 16);
  static constexpr bool kAligned = KW % (2 * GC) == 0 || (2 * GC) % KW == 0;  // a thread's value words begin with a group
  static constexpr int VG = kAligned ? (KW + 2 * GC - 1) / (2 * GC) : 2;      // groups of a thread's value words

  // what a thread has of a tile on its way
  struct stage {
    uint32_t k[KW], kr[KW], v[KW], vr[VG][8];
  };
};

template <int NC, int GC, bool WIDE, int W>
__global__ __launch_bounds__(64 * W, W == 8 || !(WIDE || NC > 4) ? 2 : 1) void k_kv4_prompt(kv4_attention_args a) {
  typedef prompt<NC, GC, WIDE, W> T;
  constexpr int NG = T::NG, D = T::D, PARTS = T::PARTS, TOKENS = T::TOKENS, SB = T::SB, KW = T::KW, ROWS = T::ROWS;
  extern __shared__ uint4 lds[];
  half8_t *const operands = (half8_t *)lds;
  uint8_t *const flags = (uint8_t *)(lds + 4 * T::kOperands);  // [2][group][token / 8], bit e: a record that is not finite

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int i = lane & 31, h = lane >> 5;
  const kv4_view &c = a.cache;
  const int rep = a.heads_per_key, head = blockIdx.x % a.key_heads;
  const int64_t unit = blockIdx.x / a.key_heads;
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
  const int all_rows = rows.count * rep, row0 = tile * ROWS;
  if (tile < 0 || row0 >= all_rows) return;  // rows before the first sequence, or a unit with none

  const int wave_row = row0 + 32 * wave, row = wave_row + i;
  const bool real = row < all_rows;
  const int t = (real ? row : 0) / rep;
  const int position = real ? rows.position + t : -1;
  const int64_t at_token = rows.first + t;
  const int at_head = head * rep + (real ? row : 0) - t * rep;

  query<2 * NC, WIDE> raw;
  raw.load(a, at_token, at_head, 8 * h, 16);
  half8_t q[PARTS][2 * NC];
  float top = kLow, sum = 0.0f;
  f32x16 o[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[n][e] = 0.0f;

  // what the workgroup's rows see, in tiles, and what the wave's do
  const int first_token = row0 / rep, last_token = (min(all_rows, row0 + ROWS) - 1) / rep;
  const int end = max(rows.position + last_token + 1, 0);
  const bool has_rows = wave_row < all_rows;
  const int low = rows.position + wave_row / rep, high = rows.position + (min(all_rows, wave_row + 32) - 1) / rep;
  int start = 0, sink_tiles = 0;
  if (a.window) {
    start = max(rows.position + first_token - a.window + 1, 0) & ~(TOKENS - 1);
    sink_tiles = (min(a.sinks, end) + TOKENS - 1) / TOKENS;
    if (sink_tiles * TOKENS >= start) start = sink_tiles = 0;
  }
  const int tiles = sink_tiles + (end > start ? (end - start + TOKENS - 1) / TOKENS : 0);
  int next = 0, stop = tiles;
  if (a.splits > 1) {
    const int chunk = a.chunk * KV4_BLOCK / TOKENS, split = blockIdx.y;
    next = (int)min((int64_t)split * chunk, (int64_t)tiles);
    if (split + 1 < a.splits) stop = (int)min((int64_t)(split + 1) * chunk, (int64_t)tiles);
  }
  auto token_of = [&](int n) { return n < sink_tiles ? n * TOKENS : start + (n - sink_tiles) * TOKENS; };

  // the thread's share of a tile: KW words of a token's key, and of eight tokens' values
  const kv4_layout lay(D, 32 * GC, 1 << c.page_shift);
  const int64_t head_offset = (int64_t)head * lay.head_bytes;
  const int page_mask = (1 << c.page_shift) - 1;
  const int kt = threadIdx.x % TOKENS, kg = threadIdx.x / TOKENS % 4, kp = threadIdx.x / TOKENS / 4;
  const int vc = threadIdx.x & 15, vj = (threadIdx.x >> 4) % (2 * T::CUT), vt = (threadIdx.x >> 4) / (2 * T::CUT);
  const code_masks masks;
  auto page_of = [&](int token) {
    const int at = token >> c.page_shift;
    return token < end && at < c.width ? kv4_list(c.table, b * c.ldtable + at) : -1;
  };
  auto page_at = [&](int page) { return c.pool + ((unsigned)page < (unsigned)c.pages ? page : 0) * c.page_stride + head_offset; };
  auto group_of = [&](int e) { return T::kAligned ? e / (2 * GC) : (vj * KW + e) / (2 * GC) - vj * KW / (2 * GC); };

  // where its words go among the operands
  const int m = (kt & 0x13) | ((kt & 8) >> 1) | ((kt & 4) << 1);
  const int k_to = ((kt >> 5) * 2 * NC + 2 * kp * KW + (kg >> 1)) * 64 + (kg & 1) * 32 + m;
  auto v_to = [&](int n) {
    return T::kOperands + (((vt >> 2) * NC + (n >> 1)) * 2 + ((vt >> 1) & 1)) * 64 + (vt & 1) * 32 + (n & 1) * 16 + vc;
  };

  auto load = [&](int token, int k_page, int v_page, typename T::stage &s) {
    const uint8_t *k = page_at(k_page);
    const int at = (token + kt) & page_mask;
    __builtin_memcpy(s.k, __builtin_assume_aligned(k + at * (D / 2) + (kg * NC + kp * KW) * 4, KW == 4 ? 16 : KW == 2 ? 8 : 4), 4 * KW);
    const uint32_t *kr = (const uint32_t *)(k + lay.key_records) + at * NG;
#pragma unroll
    for (int e = 0; e < KW; ++e) s.kr[e] = kr[KW % GC ? (kp * KW + e) / GC : kp * (KW / GC) + e / GC];
    const uint8_t *v = page_at(v_page);
    const int block = ((token + 8 * vt) & page_mask) >> 3;
    __builtin_memcpy(s.v, __builtin_assume_aligned(v + lay.value_codes + block * (4 * D) + (vc * 2 * NC + vj * KW) * 4, KW == 4 ? 16 : KW == 2 ? 8 : 4), 4 * KW);
    const int g = vj * KW / (2 * GC);
#pragma unroll
    for (int n = 0; n < T::VG; ++n)
      __builtin_memcpy(s.vr[n], __builtin_assume_aligned(v + lay.value_records + (block * NG + min(g + n, NG - 1)) * 32, 16), 32);
  };
  auto put = [&](int buffer, typename T::stage &s) {
    half8_t *const to = operands + buffer * 2 * T::kOperands;
#pragma unroll
    for (int e = 0; e < KW; ++e)
      to[k_to + e * 128] = values_of(s.k[e], masks, s.kr[e]);
    // Nothing times a value that is not finite would be NaN: it becomes 0, and the rows that see it are told by the flags
    uint32_t bad[T::VG] = {};
    half2_t some = {};
#pragma unroll
    for (int n = 0; n < T::VG; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) some = or_nan(some, last_value(s.vr[n][e], s.vr[n][4 + e]));
    if (__builtin_expect(__any(is_nan(some)), 0)) {
#pragma unroll
      for (int n = 0; n < T::VG; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int up = 0; up < 2; ++up) {
            const uint32_t part = up ? 0xFFFF0000u : 0x0000FFFFu;
            if (not_finite(as_bits(last_value(s.vr[n][e], s.vr[n][4 + e])) & part)) {
              s.vr[n][e] &= ~part;
              s.vr[n][4 + e] &= ~part;
              bad[n] |= 1u << (e + 4 * up);
            }
          }
    }
    const int g = vj * KW / (2 * GC);
    if (vc == 0)
#pragma unroll
      for (int n = 0; n < T::VG; ++n) flags[buffer * T::kFlags + min(g + n, NG - 1) * (TOKENS / 8) + vt] = (uint8_t)bad[n];
#pragma unroll
    for (int e = 0; e < KW; ++e) {
      half2_t vs[4], vb[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t x = s.vr[0][p], y = s.vr[0][4 + p];
        if (T::kAligned) {
          x = s.vr[e / (2 * GC)][p], y = s.vr[e / (2 * GC)][4 + p];
        } else if (group_of(e)) {
          x = s.vr[T::VG - 1][p], y = s.vr[T::VG - 1][4 + p];
        }
        vs[p] = as_half2(x);
        vb[p] = as_half2(y);
      }
      to[KW % 2 ? v_to(vj * KW + e) : v_to(vj * KW) + v_to(e) - v_to(0)] = values_of(s.v[e], masks, vs, vb);
    }
  };

  auto attend = [&](int buffer, int j, uint64_t there, float scale) {
#pragma clang fp contract(off)  // as in soften()
    const half8_t *const k = operands + buffer * 2 * T::kOperands, *const v = k + T::kOperands;
    const uint8_t *const f = flags + buffer * T::kFlags;
    const int flagged = lane < T::kFlags ? f[lane] : 0;
    f32x16 s[SB];
#pragma unroll
    for (int n = 0; n < SB; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[n][e] = 0.0f;
    // Products of the tile's parts in turn, so that none waits for the one before it, and operands four products ahead: left alone, the
    // compiler reads each operand when its product is due (8192 tokens 616 -> 606 us, pieces of prompts 152 -> 143).
#pragma unroll
    for (int u = 0; u < 2 * NC; ++u)
#pragma unroll
      for (int n = 0; n < SB; ++n) {
        const half8_t x = k[(n * 2 * NC + u) * 64 + lane];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) s[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, q[p][u], s[n], 0, 0, 0);
      }
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 4, 0);
#pragma unroll
    for (int i = 0; i < SB * 2 * NC - 4; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMatrix, PARTS, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedMatrix, 4 * PARTS, 0);
    uint64_t see = ~0ull;
    const uint64_t all = TOKENS == 64 ? ~0ull : 0xFFFFFFFFull;
    const bool whole = there == all && j + TOKENS - 1 <= low && (!a.window || j > high - a.window || j + TOKENS <= a.sinks);
    if (__builtin_expect(!whole, 0)) {
      // bit t: the lane's row sees token j + t
      const int d = position - j;
      see = d < 0 ? 0ull : d >= 63 ? ~0ull : (2ull << d) - 1ull;
      if (a.window) {
        const int from = d - a.window + 1, sinks = a.sinks - j;
        uint64_t in = from <= 0 ? ~0ull : from >= 64 ? 0ull : ~((1ull << from) - 1ull);
        in |= sinks <= 0 ? 0ull : sinks >= 64 ? ~0ull : (1ull << sinks) - 1ull;
        see &= in;
      }
      see &= there;
#pragma unroll
      for (int n = 0; n < SB; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int bit = 32 * n + 16 * (e >> 3) + (e & 7);  // and 8 h
          if (!((uint32_t)(see >> (8 * h + 32 * n)) >> (bit & 31) & 1u)) s[n][e] = -INFINITY;
        }
    }
    float most = s[0][0];
#pragma unroll
    for (int n = 0; n < SB; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) most = fmaxf(most, s[n][e]);
    most *= scale;
    // Product and difference are rounded once, but for bases so far from 0 that fp32 has steps of 1 and more there: then the product is
    // rounded by itself, as the largest one's is, or a power would pass a half (all of them so: 8192 rows 621 us against 612, pieces of
    // prompts 150 against 145).
    float less = top;
    if (__builtin_expect(__any(most - top > kMost || (!WIDE && fabsf(top) >= kFar)), 0)) {
      float x = raised(most, top);
      x = fmaxf(x, __shfl_xor(x, 32));
      const float f = __builtin_amdgcn_exp2f(top - x);
      less = top = x;
      sum *= f;
#pragma unroll
      for (int n = 0; n < NC; ++n) o[n] *= f;
      if (!WIDE && __any(fabsf(top) >= kFar)) {
        const float back = 1.0f / scale;
#pragma unroll
        for (int n = 0; n < SB; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[n][e] = (s[n][e] * scale - top) * back;
        less = 0.0f;
      }
    }
    half8_t p[PARTS][2 * SB];
    float of = 0.0f;
#pragma unroll
    for (int n = 0; n < SB; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = s[n][8 * u + e];
          x[e] = __builtin_amdgcn_exp2f(WIDE ? v * scale - top : __builtin_fmaf(v, scale, -less));
        }
        half2_t high[4], low[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          high[e] = half2_t{(_Float16)x[e], (_Float16)x[4 + e]};
          of = sum_of(high[e], of);
          if (WIDE) {
            low[e] = half2_t{(_Float16)(x[e] - (float)high[e].x), (_Float16)(x[4 + e] - (float)high[e].y)};
            of = sum_of(low[e], of);
          }
        }
        __builtin_memcpy(&p[0][2 * n + u], high, 16);
        if (WIDE) __builtin_memcpy(&p[PARTS - 1][2 * n + u], low, 16);
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) {
          const half8_t y = v[((n * NC + ct) * 2 + u) * 64 + lane];
#pragma unroll
          for (int w = 0; w < PARTS; ++w) o[ct] = __builtin_amdgcn_mfma_f32_32x32x16_f16(y, p[w][2 * n + u], o[ct], 0, 0, 0);
        }
      }
    sum += of;
    // the next 16 tokens' exponentials and operands between these ones' products
    constexpr int each = WIDE ? 44 : 24;  // vector instructions of 16 tokens' exponentials
    __builtin_amdgcn_sched_group_barrier(kSchedRead, NC, 0);
    __builtin_amdgcn_sched_group_barrier(kSchedVector, each, 0);
#pragma unroll
    for (int i = 0; i < 2 * SB - 1; ++i)
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) {
        __builtin_amdgcn_sched_group_barrier(kSchedMatrix, PARTS, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedVector, (each + NC - 1) / NC, 0);
      }
    __builtin_amdgcn_sched_group_barrier(kSchedMatrix, NC * PARTS, 0);
    if (__builtin_expect(__any(flagged), 0)) {
#pragma unroll
      for (int ct = 0; ct < NC; ++ct) {
        uint64_t bad = 0;
        for (int e = 0; e < TOKENS / 8; ++e) bad |= (uint64_t)f[ct / GC * (TOKENS / 8) + e] << (8 * e);
        if (bad & see) o[ct] += NAN;
      }
    }
  };

  typename T::stage s;
  if (next < stop) {
    // pages one tile further ahead than codes
    int token = token_of(next), k_page = page_of(token + kt), v_page = page_of(token + 8 * vt);
    load(token, k_page, v_page, s);
    int ahead = next + 1 < stop ? token_of(next + 1) : end, k_ahead = page_of(ahead + kt), v_ahead = page_of(ahead + 8 * vt);
    uint64_t there = __ballot((unsigned)k_page < (unsigned)c.pages);
    const float scale = raw.template halves<32>(a, real, 8 * h, 16, q[0], q[PARTS - 1]);
    put(0, s);
    __syncthreads();
    for (int buffer = 0;; buffer ^= 1) {
      const bool more = next + 1 < stop;
      const int token_now = token;
      const uint64_t there_now = TOKENS == 64 ? there : there & 0xFFFFFFFFull;
      if (more) {
        token = ahead;
        there = __ballot((unsigned)k_ahead < (unsigned)c.pages);
        load(token, k_ahead, v_ahead, s);
        ahead = next + 2 < stop ? token_of(next + 2) : end;
        k_ahead = page_of(ahead + kt);
        v_ahead = page_of(ahead + 8 * vt);
      }
      const bool none = !has_rows || token_now > high ||
                        (a.window && token_now + TOKENS - 1 <= low - a.window && token_now >= a.sinks);  // of its rows
      if (!none) attend(buffer, token_now, there_now, scale);
      if (!more) break;
      put(buffer ^ 1, s);
      __syncthreads();
      ++next;
    }
  }

  sum += __shfl_xor(sum, 32);
  if (!real) return;
  if (a.splits > 1) {
    float *to = kv4_partial(a, at_token, at_head, D);
    if (sum != 0.0f) {
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v[4] = {o[n][4 * r], o[n][4 * r + 1], o[n][4 * r + 2], o[n][4 * r + 3]};
          __builtin_memcpy(to + 32 * n + 8 * r + 4 * h, v, 16);
        }
    }
    if (h == 0) kv4_partial_end(a, at_token, at_head, D, top, sum);
    return;
  }
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int channel = 32 * n + 8 * r + 4 * h;
      if (channel >= a.dim) continue;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = o[n][4 * r + e] * f;
      if (a.out_bf16) {
        bf16_bits y[4];
        dbs_round(y, v);
        __builtin_memcpy((bf16_bits *)a.out + at_token * a.ot + at_head * a.oh + channel, y, 8);
      } else {
        __builtin_memcpy((float *)a.out + at_token * a.ot + at_head * a.oh + channel, v, 16);
      }
    }
}

template <int NC, int GC, bool WIDE, int W>
hipError_t launch_prompt(const kv4_attention_args &a, dim3 grid, hipStream_t s) {
  typedef prompt<NC, GC, WIDE, W> T;
  const auto kernel = k_kv4_prompt<NC, GC, WIDE, W>;
  if (T::kLds > 65536) {  // more than a launch gets unasked; asked for once on each device
    static std::atomic<uint64_t> asked{0};
    const uint64_t bit = a.device < 64 ? 1ull << a.device : 0ull;
    if (!(asked.load(std::memory_order_acquire) & bit)) {
      const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
      if (e != hipSuccess) return DBS_NOTE(e);
      asked.fetch_or(bit, std::memory_order_release);
    }
  }
  hipLaunchKernelGGL(kernel, grid, dim3(64 * W), T::kLds, s, a);
  return DBS_NOTE(hipGetLastError());
}

template <int NC, int GC, bool WIDE>
hipError_t launch_few(const kv4_attention_args &a, int tiles, bool share, dim3 grid, hipStream_t s) {
  constexpr int waves = kv4_waves(NC, GC, 1, WIDE);
  if constexpr (NC <= 4)
    if (tiles == 2) return launch<NC, GC, 2, WIDE>(a, grid, s);
  if constexpr (waves > 1)
    if (share) return launch<NC, GC, 1, WIDE, waves == 4 ? 8 : 4 * waves>(a, grid, s);
  return launch<NC, GC, 1, WIDE>(a, grid, s);
}

template <int NC, int GC>
hipError_t launch(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s) {
  if constexpr (NC % GC == 0) {
    if (tiles >= 4) {
      if constexpr (NC == 4 || NC == 6)
        if (tiles == 8) return launch_prompt<NC, GC, false, 8>(a, grid, s);
      return wide ? launch_prompt<NC, GC, true, 4>(a, grid, s) : launch_prompt<NC, GC, false, 4>(a, grid, s);
    }
    return wide ? launch_few<NC, GC, true>(a, tiles, share, grid, s) : launch_few<NC, GC, false>(a, tiles, share, grid, s);
  }
  return hipErrorInvalidValue;
}

template <int NC>
hipError_t launch(const kv4_attention_args &a, int tiles, bool share, bool wide, dim3 grid, hipStream_t s) {
  if (a.group == 32) return launch<NC, 1>(a, tiles, share, wide, grid, s);
  if (a.group == 64) return launch<NC, 2>(a, tiles, share, wide, grid, s);
  return launch<NC, 4>(a, tiles, share, wide, grid, s);
}

}  // namespace kv4
