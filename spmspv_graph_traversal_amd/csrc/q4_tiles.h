// The product kernel of 4-bit matrices (q4.h) on the matrix cores.
#pragma once

#include <type_traits>

#include "q4.h"

struct q4_args {
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

// How a call is cut into workgroups of `waves` waves that split the columns.
struct q4_shape {
  int token_tiles;   // of 16 tokens; 0: the kernel of one to four tokens
  int waves;
  int groups, cols;  // one to four tokens: workgroups, and columns of x in LDS at once
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

// the eight codes of a dword as bf16 16 + q: four mantissa bits under the exponent of 16, an "and or" each
DBS_DEV bf16x8 codes_operand(uint32_t w) {
  const uint32_t keep = 0x00780078u, sixteen = 0x41804180u;
  return operand((w & keep) | sixteen, ((w >> 4) & keep) | sixteen, ((w >> 8) & keep) | sixteen,
                 (__builtin_amdgcn_alignbit(w, w, 12) & keep) | sixteen);
}

// x as matrix operands: eight consecutive columns of one token per lane.  bf16 goes in as it is; fp32 is cut
// into three bf16 parts of eight mantissa bits each, which sum to it exactly.
template <class X>
struct x_part;
template <>
struct x_part<bf16_bits> {
  static constexpr int parts = 1;
  uint4 v;
  DBS_DEV void load(const bf16_bits *p) { __builtin_memcpy(&v, p, 16); }
  // columns col .. col + 7 of a row of n, zero from n on; loads of clamped addresses and no branches
  DBS_DEV void load_cut(const bf16_bits *row, int col, int n) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = row[min(col + e, n - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = col + e < n ? h[e] : 0u;
    v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
  DBS_DEV void split(bf16x8 *out) const { out[0] = operand(v.x, v.y, v.z, v.w); }
};
template <>
struct x_part<float> {
  static constexpr int parts = 3;
  float v[8];
  DBS_DEV void load(const float *p) { __builtin_memcpy(v, p, 32); }
  DBS_DEV void load_cut(const float *row, int col, int n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = row[min(col + e, n - 1)];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = col + e < n ? v[e] : 0.0f;
  }
  DBS_DEV void split(bf16x8 *out) const {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = __float_as_uint(r[2 * e]), b = __float_as_uint(r[2 * e + 1]);
        w[e] = __builtin_amdgcn_perm(b, a, 0x07060302u);  // the upper halves
        r[2 * e] -= __uint_as_float(a & 0xFFFF0000u);
        r[2 * e + 1] -= __uint_as_float(b & 0xFFFF0000u);
      }
      out[k] = operand(w[0], w[1], w[2], w[3]);
    }
  }
};

DBS_DEV bool is_finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

DBS_DEV float act_apply(int act, float g) {
  if (act == DBS_ACT_SILU) return g / (1.0f + expf(-g));
  if (act == DBS_ACT_GELU_TANH) return 0.5f * g * (1.0f + tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g)));
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
 * Both kernels below: with off = 16 + zero, a group's part of y is
 *   scale (sum (16 + q) x - off sum x),
 * so the codes go into the matrix cores as bf16 16 + q (exact, one "and or" for two of them) and sum x is a second
 * product, with ones, shared by all rows.  Both sums run in fp32 on exact products; scale and off are applied once
 * per group and row.  The first, largest part of an fp32 x keeps sums of its own: rounding next to 24 times x is
 * what loses bits, and the first part's products have few bits.  A result that is not finite is computed again
 * weight by weight.
 *
 * Split: the waves of a workgroup share its rows and take every waves-th block of 128 columns; their sums meet in LDS in a
 * fixed order.  Nothing is atomic, so results do not depend on timing.
 */

/*
 * One to four tokens.  The parts of x, of every token, are rows of one 16-row operand: bf16 token i in row i, fp32 token t
 * in rows 4t .. 4t + 2, and stand in LDS, so that the registers hold the codes of DEPTH column blocks in flight.
 * A workgroup goes through the row blocks from blockIdx.x on in steps of the grid, so that few workgroups pass over a
 * mask that leaves little.  `cols`: columns of x in LDS at once, a multiple of 128 * waves, or all of them.
 */
constexpr int kDepth = 4;
constexpr int kFewPad = 32;  // elements behind a row of x in LDS: the rows start in different banks

template <class X, int WORDS, int GPT, int MATS>
__global__ __launch_bounds__(1024) void k_q4_few(q4_args q, int cols) {
  extern __shared__ uint4 lds[];
  constexpr int P = x_part<X>::parts;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int j = lane & 15, kq = lane >> 4;
  const int tokens = q.tokens;
  bf16_bits *xs = (bf16_bits *)lds;  // [tokens * P][cols + kFewPad]
  const int pitch = cols + kFewPad;
  float *part = (float *)(lds + (tokens * P * pitch + 7) / 8);  // [waves][MATS][4][16]
  // this lane's operand row: tokens past the last one repeat it, the fourth part repeats the third; dropped
  const int arow = P == 1 ? min(j, tokens - 1) : min(j >> 2, tokens - 1) * P + min(j & 3, P - 1);
  const bf16_bits *xrow = xs + arow * pitch + 8 * kq;
  const bf16x8 ones = operand(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const X *x = (const X *)q.x;
  bool staged = false;

  for (int rt = blockIdx.x; rt < q.mt; rt += gridDim.x) {
    if (q.mask && !any_wanted(q, 0, tokens, rt * Q4_ROWS, Q4_ROWS)) {
      fill_rows(q, 0, tokens, rt * Q4_ROWS, Q4_ROWS);
      continue;
    }
    const int64_t base = (int64_t)rt * q.kt;
    f32x4 acc[MATS];
#pragma unroll
    for (int a = 0; a < MATS; ++a) acc[a] = zero;
    uint4 codes[kDepth][MATS];
    uint32_t recs[kDepth][MATS][GPT * WORDS];
    auto fetch = [&](int d, int k) {
#pragma unroll
      for (int a = 0; a < MATS; ++a) {
        codes[d][a] = ((const uint4 *)q.codes[a])[(base + k) * 64 + lane];
        __builtin_memcpy(recs[d][a], q.recs[a] + ((base + k) * Q4_ROWS + j) * (GPT * WORDS), GPT * WORDS * 4);
      }
    };
    for (int c0 = 0; c0 < q.kt * Q4_COLS; c0 += cols) {
      const int first = c0 / Q4_COLS + wave, end = min(q.kt, (c0 + cols) / Q4_COLS);
#pragma unroll
      for (int d = 0; d < kDepth; ++d)
        if (first + d * waves < end) fetch(d, first + d * waves);
      if (!staged || cols < q.kt * Q4_COLS) {
        if (staged) __syncthreads();  // the columns before these are done with
        const int width = min(cols, q.kt * Q4_COLS - c0);
        for (int u = threadIdx.x; u < tokens * (width / 8); u += blockDim.x) {
          const int t = u / (width / 8), c = u % (width / 8) * 8;
          x_part<X> v;
          const X *row = x + t * q.ldx;
          if (c0 + c + 8 <= q.n) v.load(row + c0 + c);
          else v.load_cut(row, c0 + c, q.n);
          bf16x8 p[P];
          v.split(p);
#pragma unroll
          for (int i = 0; i < P; ++i) *(bf16x8 *)(xs + (t * P + i) * pitch + c) = p[i];
        }
        staged = true;
        __syncthreads();
      }
      auto multiply = [&](int d, int k) {
        const bf16_bits *xk = xrow + (k * Q4_COLS - c0);
#pragma unroll
        for (int g = 0; g < GPT; ++g) {
          constexpr int S = 4 / GPT;  // steps of 32 columns per group
          f32x4 sum, dot[MATS];
#pragma unroll
          for (int s = 0; s < S; ++s) {
            const bf16x8 xv = *(const bf16x8 *)(xk + 32 * (g * S + s));
            sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, ones, s ? sum : zero, 0, 0, 0);
#pragma unroll
            for (int a = 0; a < MATS; ++a)
              dot[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, codes_operand(dword(codes[d][a], g * S + s)), s ? dot[a] : zero, 0, 0, 0);
          }
#pragma unroll
          for (int a = 0; a < MATS; ++a) {
            float scale, off;
            q4_record<WORDS>(recs[d][a], g, scale, off);
            if (P == 1) {
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[a][i] = fmaf(scale, fmaf(-off, sum[i], dot[a][i]), acc[a][i]);
            } else {  // smallest part first
              const float v = fmaf(-off, sum[2], dot[a][2]) + fmaf(-off, sum[1], dot[a][1]);
              acc[a][0] = fmaf(scale, v + fmaf(-off, sum[0], dot[a][0]), acc[a][0]);
            }
          }
        }
      };
      int k = first;
      for (; k + (2 * kDepth - 1) * waves < end; k += kDepth * waves) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          multiply(d, k + d * waves);
          fetch(d, k + (d + kDepth) * waves);
        }
      }
      for (; k < end; k += kDepth * waves) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
          if (k + d * waves < end) {
            multiply(d, k + d * waves);
            if (k + (d + kDepth) * waves < end) fetch(d, k + (d + kDepth) * waves);
          }
      }
    }
    // bf16: lanes kq = 0 hold token i in register i; fp32: lanes kq = t hold token t
#pragma unroll
    for (int a = 0; a < MATS; ++a) {
      float *p = part + (wave * MATS + a) * 64 + j;
      if (P == 1) {
        if (kq == 0)
#pragma unroll
          for (int i = 0; i < 4; ++i) p[16 * i] = acc[a][i];
      } else {
        p[16 * kq] = acc[a][0];
      }
    }
    __syncthreads();
    finish<X, WORDS, GPT, MATS>(q, part, waves, 4, Q4_ROWS, 0, tokens, rt * Q4_ROWS);
    __syncthreads();
  }
}

/*
 * More tokens: R x 16 rows (of each matrix) and TT x 16 tokens per workgroup; x goes from memory to the operands'
 * registers, as each wave needs its own columns of it, RING steps of 32 columns ahead, the codes one column block ahead.
 */
template <class X, int WORDS, int GPT, int MATS, int R, int TT>
__global__ __launch_bounds__(512) void k_q4_many(q4_args q) {
  extern __shared__ uint4 lds[];
  float *part = (float *)lds;  // [waves / 2][MATS][16 TT][16 R]
  constexpr int P = x_part<X>::parts, L = P > 1 ? 2 : 1;  // sums: first part, other parts
  constexpr int RING = TT * P <= 2 ? 4 : 2;
  constexpr int kRows = Q4_ROWS * R, kTokens = 16 * TT, kOut = MATS * kTokens * kRows;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int j = lane & 15, kq = lane >> 4;
  const int rt0 = blockIdx.x * R, t0 = blockIdx.y * kTokens;
  const int tokens = min(kTokens, q.tokens - t0);
  const X *x = (const X *)q.x + (int64_t)t0 * q.ldx;
  if (q.mask && !any_wanted(q, t0, tokens, rt0 * Q4_ROWS, kRows)) {
    fill_rows(q, t0, tokens, rt0 * Q4_ROWS, kRows);
    return;
  }
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const bf16x8 ones = operand(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  f32x4 acc[MATS][R][TT];
#pragma unroll
  for (int a = 0; a < MATS; ++a)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[a][r][t] = zero;
  // lanes of tokens past the last one read the last one's x; their sums are dropped
  const X *xl[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) xl[t] = x + (int64_t)min(16 * t + j, tokens - 1) * q.ldx;
  int64_t base[R];
#pragma unroll
  for (int r = 0; r < R; ++r) base[r] = (int64_t)min(rt0 + r, q.mt - 1) * q.kt;  // past the last row: dropped too

  uint4 codes[MATS][R];
  x_part<X> ring[RING][TT];
  auto fetch_codes = [&](uint4 (&to)[MATS][R], int k) {
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int r = 0; r < R; ++r) to[a][r] = ((const uint4 *)q.codes[a])[(base[r] + k) * 64 + lane];
  };
  auto fetch_x = [&](int slot, int k, int s) {
#pragma unroll
    for (int t = 0; t < TT; ++t) ring[slot][t].load(xl[t] + k * Q4_COLS + 32 * s + 8 * kq);
  };
  // Column block k, whose codes and first RING steps of x are in registers; unless it is the wave's LAST, those of block
  // `next` are fetched meanwhile.  CUT: the block that n ends in, whose x is fetched here.  Nothing in it branches: the
  // compiler would move a group's scaling behind the branch and keep its sums in registers till then.
  auto block = [&](auto last_, auto cut_, int k, int next) {
    constexpr bool LAST = decltype(last_)::value, CUT = decltype(cut_)::value;
    uint32_t recs[MATS][R][GPT * WORDS];
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int r = 0; r < R; ++r)
        __builtin_memcpy(recs[a][r], q.recs[a] + ((base[r] + k) * Q4_ROWS + j) * (GPT * WORDS), GPT * WORDS * 4);
    uint4 after[MATS][R];
    if (!LAST) fetch_codes(after, next);
    constexpr int S = 4 / GPT;  // steps of 32 columns per group
#pragma unroll
    for (int g = 0; g < GPT; ++g) {
      f32x4 sum[TT][L], dot[MATS][R][TT][L];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int step = g * S + s;
        bf16x8 xs[TT][P];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          if (CUT) {
            x_part<X> v;
            v.load_cut(xl[t], k * Q4_COLS + 32 * step + 8 * kq, q.n);
            v.split(xs[t]);
          } else {
            ring[step % RING][t].split(xs[t]);
          }
        }
        if (!CUT) {
          if (step + RING < 4) fetch_x(step % RING, k, step + RING);
          else if (!LAST) fetch_x(step % RING, next, step + RING - 4);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            f32x4 &to = sum[t][p ? L - 1 : 0];
            to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs[t][p], ones, s || p > 1 ? to : zero, 0, 0, 0);
          }
#pragma unroll
        for (int a = 0; a < MATS; ++a)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bf16x8 w = codes_operand(dword(codes[a][r], step));
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
              for (int p = 0; p < P; ++p) {
                f32x4 &to = dot[a][r][t][p ? L - 1 : 0];
                to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xs[t][p], w, s || p > 1 ? to : zero, 0, 0, 0);
              }
          }
      }
#pragma unroll
      for (int a = 0; a < MATS; ++a)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float scale, off;
          q4_record<WORDS>(recs[a][r], g, scale, off);
#pragma unroll
          for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v = fmaf(-off, sum[t][0][i], dot[a][r][t][0][i]);
              if (L > 1) v += fmaf(-off, sum[t][L - 1][i], dot[a][r][t][L - 1][i]);
              acc[a][r][t][i] = fmaf(scale, v, acc[a][r][t][i]);
            }
        }
    }
    if (!LAST) {
#pragma unroll
      for (int a = 0; a < MATS; ++a)
#pragma unroll
        for (int r = 0; r < R; ++r) codes[a][r] = after[a][r];
    }
  };
  const int whole = q.n / Q4_COLS;  // blocks that n does not end in
  if (wave < whole) {
    fetch_codes(codes, wave);
#pragma unroll
    for (int s = 0; s < RING; ++s) fetch_x(s, wave, s);
    int k = wave;
    for (; k + waves < whole; k += waves) block(std::false_type(), std::false_type(), k, k + waves);
    block(std::true_type(), std::false_type(), k, k);
  }
  if (whole < q.kt && whole % waves == wave) {
    fetch_codes(codes, whole);
    block(std::true_type(), std::true_type(), whole, whole);
  }

  // lane (kq, j), register i: token 16 t + 4 kq + i of row 16 r + j
  auto slot = [&](int a, int r, int t, int i) { return (a * kTokens + 16 * t + 4 * kq + i) * kRows + 16 * r + j; };
  const int half = (waves + 1) / 2;  // the upper half of the waves adds to the lower one first: half the LDS
  if (wave >= half) {
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[(wave - half) * kOut + slot(a, r, t, i)] = acc[a][r][t][i];
  }
  __syncthreads();
  if (wave < half) {
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float *p = part + wave * kOut + slot(a, r, t, i);
            *p = acc[a][r][t][i] + (wave + half < waves ? *p : 0.0f);
          }
  }
  __syncthreads();
  finish<X, WORDS, GPT, MATS>(q, part, half, kTokens, kRows, t0, tokens, rt0 * Q4_ROWS);
}

template <class X, int WORDS, int GPT, int MATS>
hipError_t launch_few(const q4_args &q, const q4_shape &p, hipStream_t s) {
  constexpr int P = x_part<X>::parts;
  const size_t lds = (size_t)((q.tokens * P * (p.cols + kFewPad) + 7) / 8) * 16 + (size_t)p.waves * MATS * 256;
  hipLaunchKernelGGL((k_q4_few<X, WORDS, GPT, MATS>), dim3((unsigned)p.groups), dim3(64 * p.waves), lds, s, q, p.cols);
  return DBS_NOTE(hipGetLastError());
}

template <class X, int WORDS, int GPT, int MATS, int R, int TT>
hipError_t launch_many(const q4_args &q, const q4_shape &p, hipStream_t s) {
  const dim3 grid((unsigned)((q.mt + R - 1) / R), (unsigned)((q.tokens + 16 * TT - 1) / (16 * TT)));
  const size_t lds = (size_t)((p.waves + 1) / 2) * MATS * R * TT * 1024;
  hipLaunchKernelGGL((k_q4_many<X, WORDS, GPT, MATS, R, TT>), grid, dim3(64 * p.waves), lds, s, q);
  return DBS_NOTE(hipGetLastError());
}

template <class X, int WORDS, int GPT, int MATS>
hipError_t launch_shape(const q4_args &q, const q4_shape &p, hipStream_t s) {
  if (p.token_tiles == 0) return launch_few<X, WORDS, GPT, MATS>(q, p, s);
#ifdef Q4_TUNE
  if (getenv("Q4T")) {
    int tt, r, w;
    sscanf(getenv("Q4T"), "%d,%d,%d", &tt, &r, &w);
    q4_shape z = p; z.waves = w;
    switch (tt * 10 + r) {
      case 11: return launch_many<X, WORDS, GPT, MATS, 1, 1>(q, z, s);
      case 12: return launch_many<X, WORDS, GPT, MATS, 2, 1>(q, z, s);
      case 14: return launch_many<X, WORDS, GPT, MATS, 4, 1>(q, z, s);
      case 21: return launch_many<X, WORDS, GPT, MATS, 1, 2>(q, z, s);
      case 22: return launch_many<X, WORDS, GPT, MATS, 2, 2>(q, z, s);
      case 24: return launch_many<X, WORDS, GPT, MATS, 4, 2>(q, z, s);
      case 41: return launch_many<X, WORDS, GPT, MATS, 1, 4>(q, z, s);
      case 42: return launch_many<X, WORDS, GPT, MATS, 2, 4>(q, z, s);
      case 43: return launch_many<X, WORDS, GPT, MATS, 3, 4>(q, z, s);
      case 44: return launch_many<X, WORDS, GPT, MATS, 4, 4>(q, z, s);
    }
  }
#endif
  if (p.token_tiles == 1) return launch_many<X, WORDS, GPT, MATS, 1, 1>(q, p, s);
  if (p.token_tiles == 2) return launch_many<X, WORDS, GPT, MATS, 2, 2>(q, p, s);
  return launch_many<X, WORDS, GPT, MATS, 2, 4>(q, p, s);
}

template <class X, int MATS>
hipError_t launch(const q4_args &q, int words, int gpt, const q4_shape &p, hipStream_t s) {
  if (words == 1) {
    if (gpt == 1) return launch_shape<X, 1, 1, MATS>(q, p, s);
    if (gpt == 2) return launch_shape<X, 1, 2, MATS>(q, p, s);
    return launch_shape<X, 1, 4, MATS>(q, p, s);
  }
  if (gpt == 1) return launch_shape<X, 2, 1, MATS>(q, p, s);
  if (gpt == 2) return launch_shape<X, 2, 2, MATS>(q, p, s);
  return launch_shape<X, 2, 4, MATS>(q, p, s);
}

}  // namespace q4

// each in its own source file: X x MATS
hipError_t dbs_q4_launch_bf16(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s);
hipError_t dbs_q4_launch_bf16_gated(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s);
hipError_t dbs_q4_launch_f32(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s);
hipError_t dbs_q4_launch_f32_gated(const q4_args &q, int words, int gpt, const q4_shape &shape, hipStream_t s);
