// The product kernel of 4-bit matrices (q4.h) on the matrix cores.
#pragma once

#include <atomic>
#include <type_traits>

#include "q4_shape.h"
#include "tile_kernels.h"

struct q4_args {
  int device;  // the current one
  const uint32_t *codes[2], *recs[2];  // [1]: the second matrix of a gated product
  int m, n, mt, kt, act;
  int tokens;
  const void *x;
  int64_t ldx;
  const uint32_t *mask;
  int64_t ldmask;
  float fill;
  int y_bf16;
  void *y;
  int64_t ldy;
};

namespace q4 {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

DBS_DEV bf16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 v = make_uint4(a, b, c, d);
  bf16x8 r;
  __builtin_memcpy(&r, &v, 16);
  return r;
}

// The eight codes of a dword as bf16 16 + q: four mantissa bits under the exponent of 16, an "and or" each.  The two
// constants come in registers: from literals the compiler makes two instructions.  (The empty asm only hides their value;
// an instruction in it would escape the compiler's wait states between matrix and vector instructions.)
struct code_masks {
  uint32_t keep, sixteen;
  DBS_DEV code_masks() : keep(0x00780078u), sixteen(0x41804180u) { asm("" : "+s"(keep), "+v"(sixteen)); }
};
DBS_DEV bf16x8 codes_operand(uint32_t w, const code_masks &m) {
  return operand((w & m.keep) | m.sixteen, ((w >> 4) & m.keep) | m.sixteen, ((w >> 8) & m.keep) | m.sixteen,
                 (__builtin_amdgcn_alignbit(w, w, 12) & m.keep) | m.sixteen);
}

// x on its way to the operands.  A lane takes 16 bytes of a token's row, so that adjacent lanes read adjacent bytes
// (one operand's lanes are 16 tokens: read directly, each would be a memory request of its own, 64 cycles a load
// instead of 16), and puts them into LDS as bf16: bf16 as it is, fp32 cut into three bf16 parts of eight mantissa bits,
// which sum to it exactly (bits below 2^-133, the least that bf16 holds, are left out).
template <class X>
struct x_piece;
template <>
struct x_piece<bf16_bits> {
  static constexpr int parts = 1, columns = 8;
  uint4 v;
  DBS_DEV void load(const bf16_bits *row, int col) { __builtin_memcpy(&v, row + col, 16); }
  // columns from n on are zero; loads of clamped addresses and no branches
  DBS_DEV void load_cut(const bf16_bits *row, int col, int n) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = row[min(col + e, n - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = col + e < n ? h[e] : 0u;
    v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
  // the piece was read `back` columns early, so as to end with its row: what lies past the end becomes zero.  `shift` is
  // the one value of `back` between 0 and 8 in this wave
  DBS_DEV void cut(int back, int shift) {
    const uint32_t w[8] = {v.x, v.y, v.z, v.w, 0u, 0u, 0u, 0u};
    uint32_t moved[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      moved[i] = w[i];
#pragma unroll
      for (int s = 1; s < 8; ++s)
        if (s == shift) moved[i] = s & 1 ? __builtin_amdgcn_alignbit(w[min(i + s / 2 + 1, 7)], w[i + s / 2], 16) : w[i + s / 2];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) moved[i] = back == 0 ? w[i] : back < columns ? moved[i] : 0u;
    v = make_uint4(moved[0], moved[1], moved[2], moved[3]);
  }
  // place(p): where part p of this piece goes
  template <class F>
  DBS_DEV void put(F place) const { *(uint4 *)place(0) = v; }
};
template <>
struct x_piece<float> {
  static constexpr int parts = 3, columns = 4;
  float v[4];
  DBS_DEV void load(const float *row, int col) { __builtin_memcpy(v, row + col, 16); }
  DBS_DEV void load_cut(const float *row, int col, int n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = row[min(col + e, n - 1)];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = col + e < n ? v[e] : 0.0f;
  }
  DBS_DEV void cut(int back, int shift) {
    const float w[8] = {v[0], v[1], v[2], v[3], 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float moved = w[i];
#pragma unroll
      for (int s = 1; s < 4; ++s)
        if (s == shift) moved = w[i + s];
      v[i] = back == 0 ? w[i] : back < columns ? moved : 0.0f;
    }
  }
  template <class F>
  DBS_DEV void put(F place) const {
    float r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = v[e];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t a = __float_as_uint(r[2 * e]), b = __float_as_uint(r[2 * e + 1]);
        w[e] = __builtin_amdgcn_perm(b, a, 0x07060302u);  // the upper halves
        r[2 * e] -= __uint_as_float(a & 0xFFFF0000u);
        r[2 * e + 1] -= __uint_as_float(b & 0xFFFF0000u);
      }
      *(uint2 *)place(p) = make_uint2(w[0], w[1]);
    }
  }
};

DBS_DEV bool is_finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

DBS_DEV float act_apply(int act, float g) {
  if (act == DBS_ACT_SILU) return g / (1.0f + expf(-g));
  // (1 + tanh u) / 2 as 1 / (1 + exp(-2u)): next to -1 the tanh has no bits left of the difference
  if (act == DBS_ACT_GELU_TANH) return g / (1.0f + expf(-1.5957691216057308f * (g + 0.044715f * g * g * g)));
  return g > 0.0f || g != g ? g : 0.0f;
}

// One row times one token by a whole wave, weight by weight as (code - zero) * scale.  Only for results that the
// matrix cores left infinite or NaN: there the offset of 16 meets infinities that the formula does not have.
template <int WORDS, int GPT, class X>
__device__ __noinline__ float row_dot(const uint32_t *codes, const uint32_t *recs, int kt, int n, int row, const X *x) {
  const int lane = threadIdx.x & 63, j = row & 15;
  float sum = 0.0f;
  for (int u = lane; u < kt * 16; u += DBS_WAVE) {  // dwords of the row
    const int64_t tile = (int64_t)(row >> 4) * kt + (u >> 4);
    const int s = (u >> 2) & 3, kq = u & 3;
    const int64_t col = (int64_t)(u >> 4) * Q4_COLS + 32 * s + 8 * kq;
    const uint32_t w = codes[(tile * 64 + kq * 16 + j) * 4 + s];
    float scale, off;
    q4_record<WORDS>(recs, (tile * Q4_ROWS + j) * GPT + s * GPT / 4, scale, off);
    for (int e = 0; e < 8; ++e)
      if (col + e < n) sum += (16.0f + (float)q4_code(w, e) - off) * scale * dbs_value<X>::load(x + col + e);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  return sum;
}

// LDS written by lanes of a wave and read by others of it: in order, no barrier
DBS_DEV void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

DBS_DEV uint4 bld128(brsrc_t r, uint32_t off) {
  const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int N>
DBS_DEV void load_record_words(brsrc_t r, uint32_t off, uint32_t *to) {
  if (N == 1) to[0] = bld32(r, off);
  else if (N == 2) {
    const uint64_t v = bld64(r, off);
    to[0] = (uint32_t)v;
    to[N - 1] = (uint32_t)(v >> 32);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = bld128(r, off + 16 * i);
      to[4 * i] = v.x;
      to[4 * i + 1] = v.y;
      to[4 * i + 2] = v.z;
      to[4 * i + 3] = v.w;
    }
  }
}

DBS_DEV uint32_t dword(const uint4 &v, int s) { return s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w; }

DBS_DEV void store(const q4_args &q, int64_t at, float v) {
  if (q.y_bf16) ((bf16_bits *)q.y)[at] = dbs_value<bf16_bits>::of(v);
  else ((float *)q.y)[at] = v;
}

// whether any of `tokens` tokens from t0 on wants any of the `rows` rows from row0 on (rows a multiple of 16, row0 of
// rows): the same answer in every lane
DBS_DEV bool any_wanted(const q4_args &q, int t0, int tokens, int row0, int rows) {
  const int lane = threadIdx.x & 63, words = (rows + 31) / 32;
  uint32_t any = 0u;
  for (int i = lane; i < tokens * words; i += DBS_WAVE) {
    const int first = row0 + 32 * (i % words);  // 16 rows: the upper or lower half of a word
    if (first < q.m) {
      const uint32_t w = q.mask[(int64_t)(t0 + i / words) * q.ldmask + (first >> 5)] >> (first & 31);
      const int count = min(min(32, q.m - first), rows - 32 * (i % words));
      any |= count < 32 ? w & ((1u << count) - 1u) : w;
    }
  }
  return __ballot(any != 0u) != 0ull;
}

DBS_DEV void fill_rows(const q4_args &q, int t0, int tokens, int row0, int rows) {
  for (int i = threadIdx.x; i < tokens * rows; i += blockDim.x) {
    const int row = row0 + i % rows;
    if (row < q.m) store(q, (int64_t)(t0 + i / rows) * q.ldy + row, q.fill);
  }
}

// The outputs of a workgroup from its `parts` partial sums part[parts][MATS][stride tokens][rows]: added in order,
// masked, recomputed where not finite, activated, stored.
template <class X, int WORDS, int GPT, int MATS>
DBS_DEV void finish(const q4_args &q, const float *part, int parts, int stride, int rows, int t0, int tokens, int row0) {
  const int lane = threadIdx.x & 63, out_size = MATS * stride * rows;
  const X *x = (const X *)q.x + (int64_t)t0 * q.ldx;
  // whole waves go through the outputs together: row_dot needs all lanes
  for (int i0 = threadIdx.x - lane; i0 < tokens * rows; i0 += blockDim.x) {
    const int i = i0 + lane, token = i / rows, row = row0 + i % rows;
    const bool out = i < tokens * rows && row < q.m;
    bool wanted = out;
    if (q.mask && out) wanted = (q.mask[(int64_t)(t0 + token) * q.ldmask + (row >> 5)] >> (row & 31)) & 1u;
    float v[MATS];
#pragma unroll
    for (int a = 0; a < MATS; ++a) {
      v[a] = 0.0f;
      if (wanted) {
        for (int w = 0; w < parts; ++w) v[a] += part[w * out_size + (a * stride + token) * rows + i % rows];
      }
      unsigned long long again = __ballot(!is_finite(v[a]));
      while (again) {
        const int l = __ffsll((long long)again) - 1;
        again &= again - 1;
        const int li = i0 + l;
        const float s = row_dot<WORDS, GPT, X>(q.codes[a], q.recs[a], q.kt, q.n, row0 + li % rows,
                                               x + (int64_t)(li / rows) * q.ldx);
        if (lane == l) v[a] = s;
      }
    }
    if (out) store(q, (int64_t)(t0 + token) * q.ldy + row,
                   !wanted ? q.fill : MATS == 2 ? act_apply(q.act, v[0]) * v[MATS - 1] : v[0]);
  }
}

/*
 * y_t = W x_t for a workgroup's 16 R RW rows (of MATS matrices; RW waves share x) and TOKENS tokens: tiles of 16, of which 8
 * leave the upper half as it is in LDS (its sums are dropped), or up to four (FEW).
 *
 * Mathematics: with off = 16 + zero, a group's part of y is
 *   scale (sum (16 + q) x - off sum x),
 * so the codes go into the matrix cores as bf16 16 + q (exact, one "and or" for two of them) and sum x is a second
 * product, with ones, shared by all rows.  Both sums run in fp32 on exact products; scale and off are applied once
 * per group and row.  The first, largest part of an fp32 x keeps sums of its own: rounding next to 24 times x is
 * what loses bits, and the first part's products have few bits.  A result that is not finite is computed again
 * weight by weight.
 *
 * What bounds it (times of a graph of launches, 1.95 us of each being the launch; a copy reaches 4.9 TB/s here, reads 5.5).
 *   One token, memory and the length of a wave's chain: 4096 x 4096 4.0 us from the Infinity Cache, 5.0 where every call reads
 *   other codes, 11008 x 4096 6.5 (23.3 MB), two of these gated 11.2, other codes every time 13.9 (46.6 MB, 3.9 TB/s without the
 *   launch).
 *   Many tokens, instruction issue: a vector instruction takes four cycles of a SIMD, the unpacking of an operand (seven of
 *   them) as long as the products of two token tiles, and the two kinds hardly overlap.  11008 x 4096, 64 tokens, 17.8 us (other
 *   codes 19.3), of which vector instructions issue for 7.1, the codes being unpacked again for every 16 tokens, and the matrix
 *   cores run for 3.4, a third of it for the products with ones, which each wave makes for itself; the rest is the launch, and
 *   three rounds of workgroups for the work of 2.7.  28672 x 8192 58 us, 520 TFLOP/s.
 *   fp32 x, 5461 x 2001 gated, 24 tokens, 13.6 us: three products and the cutting of x in place of one, half the time; 172
 *   workgroups leave a third of the compute units idle.
 *
 * Split: `splits` waves share the rows of a row wave and take every splits-th block of 128 columns; their sums meet in LDS
 * in a fixed order.  Nothing is atomic, so results do not depend on timing.
 *
 * x: each wave takes its own columns through LDS of its own (no barrier), rows of 256 bytes whose 16-byte pieces are
 * rotated by the row (exclusive or) so that neither side meets bank conflicts.  FEW: the parts of an fp32 x are rows of one
 * operand, token t's in rows 4t .. 4t + 2.
 *
 * Loads come back in order, and x (from L2) must not queue behind codes (from memory) of a later block.  So two blocks are in
 * flight: when block b is used up, its registers take x and codes of block b + 2, in this order.  Blocks past a wave's last
 * are out of range of the codes' buffer descriptor and read nothing.  Streaming loads of the codes (past the caches) were
 * slower: gated 12.1 us against 11.1.
 */
template <class X, int MATS, int R, int TOKENS, int RW>
struct tiling {
  static constexpr bool FEW = TOKENS == 4;
  static constexpr int TT = TOKENS < 16 ? 1 : TOKENS / 16;
  static constexpr int P = x_piece<X>::parts;
  static constexpr int kOps = FEW ? 1 : P;               // operands of a token tile and step
  static constexpr int kSums = kOps > 1 ? 2 : 1;         // sums: first part, other parts
  static constexpr int kRowsPerLoad = 64 * x_piece<X>::columns / Q4_COLS;
  static constexpr int kTokens = TOKENS;
  static constexpr int kLoads = kTokens / kRowsPerLoad / RW;  // of a column block's x, per wave
  static constexpr int kPlane = TT * 16 * 256;           // bytes of a part of x
  static constexpr int kBuffers = RW > 1 ? 2 : 1;
  static constexpr int kLds = kBuffers * kOps * kPlane;  // per split
  static constexpr int kDepth = 2;                // column blocks in flight
  // sixteen waves may use 128 registers each, twelve 168, eight 256
  static constexpr int kThreads = FEW || MATS * R * TT * kOps <= 2 ? 1024 : MATS * R * TT == 1 ? 768 : 512;
  static_assert(kLoads >= 1, "");
  // as many of the splits as registers and LDS allow
  static int fitting(int splits) {
    while (splits * kLds > 160 * 1024 || 64 * splits * RW > kThreads) splits /= 2;
    return splits;
  }
};

template <class X, int WORDS, int GPT, int MATS, int R, int TOKENS, int RW>
__global__ __launch_bounds__((tiling<X, MATS, R, TOKENS, RW>::kThreads)) void k_q4(q4_args q) {
  extern __shared__ uint4 lds[];
  typedef tiling<X, MATS, R, TOKENS, RW> T;
  constexpr bool FEW = T::FEW;
  constexpr int TT = T::TT;
  constexpr int kRec = GPT * WORDS, kTokens = T::kTokens, rows = Q4_ROWS * R * RW;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, split = wave / RW, splits = (blockDim.x >> 6) / RW;
  const int j = lane & 15, kq = lane >> 4;
  // Workgroups go to the eight dies in turn, and each die has an L2 of its own: the token blocks (y) of one row group are a
  // multiple of eight apart, so that they run on one die at one time and the codes come from memory once.
  const unsigned first = (blockIdx.z * gridDim.x + blockIdx.x) * rows;
  if (first >= (unsigned)q.m) return;
  const int row0 = (int)first, rt0 = row0 / Q4_ROWS + rw * R, t0 = blockIdx.y * kTokens;
  const int tokens = min(kTokens, q.tokens - t0);
  const X *x = (const X *)q.x + (int64_t)t0 * q.ldx;
  if (q.mask && !any_wanted(q, t0, tokens, row0, rows)) {
    fill_rows(q, t0, tokens, row0, rows);
    return;
  }
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const bf16x8 ones = operand(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  const code_masks masks;
  f32x4 acc[MATS][R][TT];
#pragma unroll
  for (int a = 0; a < MATS; ++a)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[a][r][t] = zero;

  // load i of this row wave takes its lanes' pieces of tokens kRowsPerLoad (RW i + rw) + lane / kPieces; tokens past the
  // last one repeat it, their sums are dropped
  constexpr int kPieces = 64 / T::kRowsPerLoad;
  const int piece = lane % kPieces;
  const X *from[T::kLoads];
  int to[T::kLoads];
  char *const xlds = (char *)lds + split * T::kLds;
#pragma unroll
  for (int i = 0; i < T::kLoads; ++i) {
    const int token = T::kRowsPerLoad * (RW * i + rw) + lane / kPieces;
    from[i] = x + (int64_t)min(token, tokens - 1) * q.ldx + piece * x_piece<X>::columns;
    // FEW fp32: part p of a token in row 4 token + p; otherwise parts are kPlane bytes apart
    const int row = FEW && T::P > 1 ? token * 4 : token, chunk = piece * x_piece<X>::columns / 8;
    to[i] = row * 256 + ((chunk ^ row) & 15) * 16 + piece * x_piece<X>::columns % 8 * 2;
  }
  const int whole = q.n / Q4_COLS;  // column blocks that n does not end in
  brsrc_t rc[MATS][R], rr[MATS][R];
#pragma unroll
  for (int a = 0; a < MATS; ++a)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t first = (int64_t)min(rt0 + r, q.mt - 1) * q.kt;  // past the last row block: dropped too
      rc[a][r] = make_rsrc((const char *)q.codes[a] + first * Q4_TILE_BYTES, (uint64_t)q.kt * Q4_TILE_BYTES);
      rr[a][r] = make_rsrc(q.recs[a] + first * (Q4_ROWS * kRec), (uint64_t)q.kt * (Q4_ROWS * kRec * 4));
    }

  constexpr int D = T::kDepth;
  uint4 codes[D][MATS][R];
  uint32_t recs[D][MATS][R][kRec];
  x_piece<X> xr[D][T::kLoads];
  auto fetch_codes = [&](int d, int k, int end) {
    const uint32_t oc = q4_code_offset(k, end, lane), orec = q4_record_offset(k, end, j, kRec);
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        codes[d][a][r] = bld128(rc[a][r], oc);
        load_record_words<kRec>(rr[a][r], orec, recs[d][a][r]);
      }
  };
  auto put_x = [&](int d) {
    char *at = xlds + (RW > 1 ? d % 2 * (T::kOps * T::kPlane) : 0);
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i)
      xr[d][i].put([&](int p) { return FEW ? at + (to[i] ^ p << 4) + p * 256 : at + to[i] + p * T::kPlane; });
  };
  // The products of one column block.  Nothing in it branches: the compiler would move a group's scaling behind the branch
  // and keep its sums in registers till then.
  auto multiply = [&](int d) {
    constexpr int S = 4 / GPT;  // steps of 32 columns per group
    const char *at = xlds + (RW > 1 ? d % 2 * (T::kOps * T::kPlane) : 0) + j * 256;
#pragma unroll
    for (int g = 0; g < GPT; ++g) {
      f32x4 sum[TT][T::kSums], dot[MATS][R][TT][T::kSums];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int step = g * S + s;
        bf16x8 xs[TT][T::kOps];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int p = 0; p < T::kOps; ++p) {
            xs[t][p] = *(const bf16x8 *)(at + p * T::kPlane + t * 4096 + (((4 * step + kq) ^ j) & 15) * 16);
            f32x4 &into = sum[t][p ? T::kSums - 1 : 0];
            into = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs[t][p], ones, s || p > 1 ? into : zero, 0, 0, 0);
          }
#pragma unroll
        for (int a = 0; a < MATS; ++a)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bf16x8 w = codes_operand(dword(codes[d][a][r], step), masks);
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
              for (int p = 0; p < T::kOps; ++p) {
                f32x4 &into = dot[a][r][t][p ? T::kSums - 1 : 0];
                into = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs[t][p], w, s || p > 1 ? into : zero, 0, 0, 0);
              }
          }
      }
#pragma unroll
      for (int a = 0; a < MATS; ++a)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float scale, off;
          q4_record<WORDS>(recs[d][a][r], g, scale, off);
          if (FEW && T::P > 1) {  // registers 0 .. 2 hold the parts' sums; smallest first
            const f32x4 d = dot[a][r][0][0], m = sum[0][0];
            const float low = fmaf(-off, m[2], d[2]) + fmaf(-off, m[1], d[1]);
            acc[a][r][0][0] = fmaf(scale, low + fmaf(-off, m[0], d[0]), acc[a][r][0][0]);
          } else {
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float v = fmaf(-off, sum[t][0][i], dot[a][r][t][0][i]);
                if (T::kSums > 1) v += fmaf(-off, sum[t][T::kSums - 1][i], dot[a][r][t][T::kSums - 1][i]);
                acc[a][r][t][i] = fmaf(scale, v, acc[a][r][t][i]);
              }
          }
        }
    }
  };
  // A block from its registers: x through LDS, for this wave or for all that share it.  Two buffers there: who writes one
  // again has passed a barrier since its readers were done.
  auto block = [&](int d) {
    put_x(d);
    if (RW > 1) dbs_barrier_lds();
    else wave_fence();
    multiply(d);
    if (RW == 1) wave_fence();
  };
  // All blocks of this wave.  CUT: n ends within the last of the columns' blocks; there, pieces that would pass the end are
  // read `back` columns early, and cut afterwards.  (One code for both would cost whole columns 3 %.)
  auto all_blocks = [&](auto cut) {
    constexpr bool CUT = decltype(cut)::value;
    const int back = max((whole * Q4_COLS + (piece + 1) * x_piece<X>::columns) - q.n, 0);
    const int shift = (x_piece<X>::columns - q.n % x_piece<X>::columns) % x_piece<X>::columns;
    auto fetch = [&](int d, int k) {
      __builtin_amdgcn_sched_barrier(0);  // in the order in which they are used
      const int kx = min(k, q.kt - 1);
      const int at = kx * Q4_COLS - (CUT && kx == whole ? back : 0);
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i) xr[d][i].load(from[i], at);
      __builtin_amdgcn_sched_barrier(0);
      fetch_codes(d, k, q.kt);
      __builtin_amdgcn_sched_barrier(0);
    };
    // Row waves meet at barriers, so all splits go the same number of rounds; rounds without a block multiply by zero.
    const int rounds = (q.kt - (RW > 1 ? 0 : split) + splits - 1) / splits;
    int k = split;
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, k + d * splits);
    // one way through each turn: where paths with and without loads met, the compiler would wait for all of them
    const int turns = (rounds - 1) / D;
    for (int i = 0; i < turns; ++i) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        block(d);
        k += splits;
        fetch(d, k + (D - 1) * splits);
      }
    }
    // the last block of the columns is the last of its split
    const int left = rounds - turns * D;
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (d == left) break;
      if (CUT && k + d * splits == whole) {
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) xr[d][i].cut(back, shift);
      }
      block(d);
    }
  };
  if (whole == 0) {  // less than a column block: n may be too short for a wide load
    fetch_codes(0, split, q.kt);
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i)
      xr[0][i].load_cut(from[i] - piece * x_piece<X>::columns, piece * x_piece<X>::columns, q.n);
    block(0);
  } else if (whole == q.kt) {
    all_blocks(std::false_type());
  } else {
    all_blocks(std::true_type());
  }

  // part[splits / 2][MATS][kTokens][rows], over the x of before.  Lane (kq, j), register i: token 16 t + 4 kq + i of row
  // 16 r + j; FEW bf16: lanes kq = 0 only, FEW fp32: token kq in register 0
  __syncthreads();
  float *part = (float *)lds;
  const int out_size = MATS * kTokens * rows, half = (splits + 1) / 2;
  auto each = [&](auto &&use) {
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (FEW && T::P > 1 && i) continue;
            if (FEW && T::P == 1 && kq) continue;
            if (TOKENS == 8 && kq > 1) continue;
            const int token = FEW ? (T::P > 1 ? kq : i) : 16 * t + 4 * kq + i;
            use((a * kTokens + token) * rows + 16 * (rw * R + r) + j, acc[a][r][t][i]);
          }
  };
  // the upper half of the splits adds to the lower one first: half the LDS
  if (split >= half) each([&](int at, float v) { part[(split - half) * out_size + at] = v; });
  __syncthreads();
  if (split < half)
    each([&](int at, float v) {
      float *p = part + split * out_size + at;
      *p = v + (split + half < splits ? *p : 0.0f);
    });
  __syncthreads();
  finish<X, WORDS, GPT, MATS>(q, part, half, kTokens, rows, t0, tokens, row0);
}

template <class X, int WORDS, int GPT, int MATS, int R, int TOKENS, int RW>
hipError_t launch_tiles(const q4_args &q, int splits, hipStream_t s) {
  typedef tiling<X, MATS, R, TOKENS, RW> T;
  constexpr int rows = R * RW;
  splits = T::fitting(splits);
  const auto kernel = k_q4<X, WORDS, GPT, MATS, R, TOKENS, RW>;
  const unsigned groups = (unsigned)((q.mt + rows - 1) / rows), eights = (groups + 7) / 8, wide = (eights + 65534) / 65535;
  const dim3 grid(8 * wide, (unsigned)((q.tokens + T::kTokens - 1) / T::kTokens), (eights + wide - 1) / wide);
  const size_t parts = (size_t)((splits + 1) / 2) * MATS * rows * Q4_ROWS * T::kTokens * 4;
  const size_t xs = (size_t)splits * T::kLds, lds = parts > xs ? parts : xs;
  if (lds > 65536) {  // more than a launch gets unasked; asked for once on each device
    static std::atomic<uint64_t> asked{0};
    const uint64_t bit = q.device < 64 ? 1ull << q.device : 0ull;
    if (!(asked.load(std::memory_order_acquire) & bit)) {
      const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
      if (e != hipSuccess) return DBS_NOTE(e);
      asked.fetch_or(bit, std::memory_order_release);
    }
  }
  hipLaunchKernelGGL(kernel, grid, dim3(64 * splits * RW), lds, s, q);
  return DBS_NOTE(hipGetLastError());
}

// a kernel's parameters
template <class X, int WORDS, int GPT, int MATS, int R, int TOKENS, int RW>
struct form {
  static hipError_t launch(const q4_args &q, int splits, hipStream_t s) {
    return launch_tiles<X, WORDS, GPT, MATS, R, TOKENS, RW>(q, splits, s);
  }
};

// use() of the kernel of a shape
template <class X, int WORDS, int GPT, int MATS, int TOKENS, class F>
hipError_t with_rows(const q4_shape &p, const F &use) {
  if (p.rows == 1) return use(form<X, WORDS, GPT, MATS, 1, TOKENS, 1>());
  if (p.rows == 2) {
    if constexpr (MATS == 1) return use(form<X, WORDS, GPT, MATS, 2, TOKENS, 1>());
    else return use(form<X, WORDS, GPT, MATS, 1, TOKENS, 2>());
  }
  if (p.rows == 4) {
    if constexpr (MATS == 1) return use(form<X, WORDS, GPT, MATS, 2, TOKENS, 2>());
    // (of eight bf16 tokens, four waves would not have a load each)
    else return use(form<X, WORDS, GPT, MATS, 1, sizeof(X) == 2 ? 16 : TOKENS, 4>());
  }
  if constexpr (MATS == 1 && sizeof(X) == 4) {
    if (p.rows == 8) return use(form<X, WORDS, GPT, MATS, 2, TOKENS, 4>());
  }
  return hipErrorInvalidValue;
}

template <class X, int WORDS, int GPT, int MATS, class F>
hipError_t with_shape(const q4_shape &p, const F &use) {
  if (p.tokens == 4) {
    if constexpr (MATS == 1) {
      if (p.rows == 2) return use(form<X, WORDS, GPT, MATS, 2, 4, 1>());
    }
    return use(form<X, WORDS, GPT, MATS, 1, 4, 1>());
  }
  if (p.tokens == 32) {
    if constexpr (sizeof(X) == 2) return use(form<X, WORDS, GPT, MATS, MATS == 1 ? 2 : 1, 32, 4>());
    return hipErrorInvalidValue;
  }
  if (p.tokens == 8) return with_rows<X, WORDS, GPT, MATS, 8>(p, use);
  return with_rows<X, WORDS, GPT, MATS, 16>(p, use);
}

template <class X, int MATS, class F>
hipError_t with_form(int words, int gpt, const q4_shape &p, const F &use) {
  if (words == 1) {
    if (gpt == 1) return with_shape<X, 1, 1, MATS>(p, use);
    if (gpt == 2) return with_shape<X, 1, 2, MATS>(p, use);
    return with_shape<X, 1, 4, MATS>(p, use);
  }
  if (gpt == 1) return with_shape<X, 2, 1, MATS>(p, use);
  if (gpt == 2) return with_shape<X, 2, 2, MATS>(p, use);
  return with_shape<X, 2, 4, MATS>(p, use);
}

template <class X, int MATS>
hipError_t launch(const q4_args &q, int words, int gpt, const q4_shape &p, hipStream_t s) {
  return with_form<X, MATS>(words, gpt, p, [&](auto kernel) { return kernel.launch(q, p.splits, s); });
}

}  // namespace q4

// each in its own source file: X x MATS
hipError_t dbs_q4_launch_bf16(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s);
hipError_t dbs_q4_launch_bf16_gated(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s);
hipError_t dbs_q4_launch_f32(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s);
hipError_t dbs_q4_launch_f32_gated(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s);
