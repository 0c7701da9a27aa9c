// Root mean square norms of query and key heads with their rotary positions (dbs_norm_rope).
#include "rope.h"

#include <math.h>

namespace {

struct norm_part {
  const void *x;
  int64_t xt, xh;
  void *out;
  int64_t ot, oh;
  const void *weight;
};
struct norm_args {
  int tokens, heads, first_heads, head_dim, rot_dim;  // heads: of both parts
  bool weight_bf16;
  const int32_t *pos;
  const double *freq;
  float scale, eps;
  norm_part part[2];
};

/*
 * Mathematics: y = turn(w * x * r), r = 1 / sqrt(mean(x^2) + eps), per head, all in fp32; pairs of the first rot_dim elements turn
 * as in dbs_rope.  x is read once and kept in registers while its squares are summed: `lanes` lanes hold a head, each
 * UNITS units of W pairs or W elements behind them, the two halves of a pair in one lane, so the sum of squares is the only
 * exchange.  Queries and keys share a token's sines and one launch.
 *
 * One workgroup per token and `per` heads.  Bound by memory for a prompt: 8192 tokens of 40 heads of 128 bf16 34 us, 168 MB at
 * 4.9 TB/s, with eight waves a SIMD (40 with six) and values rounded in pairs; weights asked for early cost registers and time
 * (41).  A token takes the launch and one chain of loads, 3.8 us.
 */
template <class X, class Y, int W, bool INTERLEAVED, int UNITS>
__global__ __launch_bounds__(512, UNITS == 1 ? 8 : 1) void k_norm_rope(norm_args n, int per, int lanes) {
  static constexpr bool kMixed = INTERLEAVED && W > 1;  // 2 W neighbours, of which those from rot_dim on do not turn
  __shared__ float2 turn[DBS_ROPE_MAX_DIM / 2];
  const int64_t t = blockIdx.x;
  const int p = n.pos[t];
  if (p < 0) return;
  const int half = n.rot_dim / 2, h0 = blockIdx.y * per, count = min(per, n.heads - h0);
  const int turned = half / W, units = rope_units<W, INTERLEAVED>(n.head_dim, n.rot_dim);
  const int lane = threadIdx.x & (lanes - 1), step = blockDim.x / lanes;

  X a[UNITS][W], b[UNITS][W];
  auto paired = [&](int i) { return kMixed || i < turned; };
  auto at_a = [&](int i) { return INTERLEAVED && paired(i) ? 2 * W * i : paired(i) ? W * i : 2 * half + W * (i - turned); };
  auto at_b = [&](int i) { return INTERLEAVED ? 2 * W * i + W : half + W * i; };
  auto load = [&](int h) {
    const norm_part &s = n.part[h >= n.first_heads];
    const X *x = (const X *)s.x + t * s.xt + (h >= n.first_heads ? h - n.first_heads : h) * s.xh;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int i = lane + u * lanes;
      if (i >= units) break;
      __builtin_memcpy(a[u], x + at_a(i), sizeof a[u]);
      if (paired(i)) __builtin_memcpy(b[u], x + at_b(i), sizeof b[u]);
    }
  };
  auto weight = [&](const void *w, int at, float (&v)[W]) {
    if (!w) {
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = 1.0f;
    } else if (n.weight_bf16) {
      bf16_bits h[W];
      __builtin_memcpy(h, (const bf16_bits *)w + at, sizeof h);
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = bf16_to_f32(h[e]);
    } else {
      __builtin_memcpy(v, (const float *)w + at, sizeof v);
    }
  };
  auto finish = [&](int h) {
    const norm_part &s = n.part[h >= n.first_heads];
    Y *y = (Y *)s.out + t * s.ot + (h >= n.first_heads ? h - n.first_heads : h) * s.oh;
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int i = lane + u * lanes;
      if (i >= units) break;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float v = dbs_value<X>::load(&a[u][e]);
        sum += v * v;
      }
      if (paired(i))
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float v = dbs_value<X>::load(&b[u][e]);
          sum += v * v;
        }
    }
    for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor(sum, o);
    const float r = 1.0f / sqrtf(sum / n.head_dim + n.eps);
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int i = lane + u * lanes;
      if (i >= units) break;
      float wa[W], wb[W], va[W], vb[W];
      Y oa[W], ob[W];
      weight(s.weight, at_a(i), wa);
#pragma unroll
      for (int e = 0; e < W; ++e) va[e] = dbs_value<X>::load(&a[u][e]) * r * wa[e];
      if (!paired(i)) {
        dbs_round(oa, va);
        rope_write(y + at_a(i), oa);
        continue;
      }
      weight(s.weight, at_b(i), wb);
#pragma unroll
      for (int e = 0; e < W; ++e) vb[e] = dbs_value<X>::load(&b[u][e]) * r * wb[e];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const int ka = INTERLEAVED ? 2 * e : e, kb = INTERLEAVED ? 2 * e + 1 : W + e;  // within a, b
        float &ra = ka < W ? va[ka % W] : vb[ka % W], &rb = kb < W ? va[kb % W] : vb[kb % W];
        if (!kMixed || W * i + e < half) {
          const float2 w = turn[W * i + e];
          const float x0 = ra, x1 = rb;
          ra = x0 * w.x - x1 * w.y;
          rb = x0 * w.y + x1 * w.x;
        }
      }
      dbs_round(oa, va);
      dbs_round(ob, vb);
      rope_write(y + at_a(i), oa);
      rope_write(y + at_b(i), ob);
    }
  };

  int h = threadIdx.x / lanes;
  if (h < count) load(h0 + h);
  for (int i = threadIdx.x; i < half; i += blockDim.x) turn[i] = rope_turn(p, n.freq[i], n.scale, 1.0f);
  dbs_barrier_lds();
  if (h < count) finish(h0 + h);
  for (h += step; h < count; h += step) {
    load(h0 + h);
    finish(h0 + h);
  }
}

template <class X, class Y, int W, bool INTERLEAVED>
dbs_status launch_norm(const norm_args &n, hipStream_t s) {
  const int units = rope_units<W, INTERLEAVED>(n.head_dim, n.rot_dim);
  int lanes = 1;
  while (lanes < units && lanes < 64) lanes <<= 1;
  // as in dbs_rope: all heads of a token share its sines, few tokens are spread over workgroups of 256 lanes by head
  int per = n.heads;
  if (n.tokens < 512) per = 256 / lanes;
  if (per > n.heads) per = n.heads;
  if (per < (n.heads + 65534) / 65535) per = (n.heads + 65534) / 65535;  // the grid's limit
  const int64_t all = (int64_t)per * lanes, rounds = (all + 511) / 512;
  const int threads = (int)((all + rounds * 64 - 1) / (rounds * 64)) * 64;
  const int most = (int)(0x7FFFFFFF / threads);  // a launch's lanes are counted in 32 bits
  const auto run = units <= 64 ? k_norm_rope<X, Y, W, INTERLEAVED, 1> : k_norm_rope<X, Y, W, INTERLEAVED, DBS_ROPE_MAX_DIM / 64 / W>;
  for (int t = 0;; t += most) {
    const int count = n.tokens - t < most ? n.tokens - t : most;
    norm_args now = n;
    now.pos += t;
    for (norm_part &p : now.part) {
      p.x = (const X *)p.x + t * p.xt;
      p.out = (Y *)p.out + t * p.ot;
    }
    hipLaunchKernelGGL(run, dim3((unsigned)count, (unsigned)((n.heads + per - 1) / per)), dim3(threads), 0, s, now, per, lanes);
    if (DBS_NOTE(hipGetLastError()) != hipSuccess) return DBS_ERR_DEVICE;
    if (count == n.tokens - t) return DBS_OK;
  }
}

// the widest units that the sizes are made of, up to 16 bytes a lane (as in dbs_rope)
template <class X, class Y>
dbs_status launch_norm(const norm_args &n, bool interleaved, hipStream_t s) {
  constexpr int most = 16 / (sizeof(X) > sizeof(Y) ? sizeof(X) : sizeof(Y));
  if (interleaved) {
    if (n.head_dim % most == 0) return launch_norm<X, Y, most / 2, true>(n, s);
    if (most == 8 && n.head_dim % 4 == 0) return launch_norm<X, Y, 2, true>(n, s);
    return launch_norm<X, Y, 1, true>(n, s);
  }
  const int width = n.rot_dim / 2 | (n.head_dim - n.rot_dim);
  if (width % most == 0) return launch_norm<X, Y, most, false>(n, s);
  if (most == 8 && width % 4 == 0) return launch_norm<X, Y, 4, false>(n, s);
  if (width % 2 == 0) return launch_norm<X, Y, 2, false>(n, s);
  return launch_norm<X, Y, 1, false>(n, s);
}

// whether heads of two sets of the same tokens may share a byte, bytes between a token's heads included
bool parts_meet(const dbs_rows &a, const dbs_rows &b) { return dbs_rows_meet(a.joined(), b.joined()); }

}  // namespace

extern "C" dbs_status dbs_norm_rope(int32_t tokens, int32_t head_dim, int32_t rot_dim, dbs_rope_layout layout, const int32_t *pos,
                                    const double *freq, float scale, float eps, const dbs_norm_part *parts, int32_t count,
                                    dbs_dtype x_dtype, dbs_dtype out_dtype, dbs_dtype weight_dtype, void *stream) {
  if (tokens < 0 || head_dim < 1 || rot_dim < 0 || rot_dim > head_dim || (rot_dim & 1) || !parts || count < 1 || count > 2)
    return DBS_ERR_INVALID_ARG;
  if (layout != DBS_ROPE_HALF && layout != DBS_ROPE_INTERLEAVED) return DBS_ERR_INVALID_ARG;
  if (!dbs_is_vector_dtype(x_dtype) || !dbs_is_vector_dtype(out_dtype) || !dbs_is_vector_dtype(weight_dtype)) return DBS_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps)) return DBS_ERR_INVALID_ARG;
  int64_t heads = 0;
  for (int i = 0; i < count; ++i) {
    if (parts[i].heads < 0) return DBS_ERR_INVALID_ARG;
    heads += parts[i].heads;
  }
  if (head_dim > DBS_ROPE_MAX_DIM || heads * head_dim > DBS_ROPE_MAX_ELEMENTS) return DBS_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0) return DBS_OK;
  if (!pos || (rot_dim > 0 && !freq)) return DBS_ERR_INVALID_ARG;
  const __int128 xs = dbs_vector_size(x_dtype), os = dbs_vector_size(out_dtype);
  const int64_t weight_bytes = head_dim * dbs_vector_size(weight_dtype);
  dbs_rows from[2], to[2];
  for (int i = 0; i < count; ++i) {
    const dbs_norm_part &p = parts[i];
    if (p.heads == 0) continue;
    if (!p.x || !p.out) return DBS_ERR_INVALID_ARG;
    const int64_t xt = p.x_token_stride, xh = p.x_head_stride, ot = p.out_token_stride, oh = p.out_head_stride;
    if (!dbs_rows_apart(tokens, ot, p.heads, oh, head_dim) && !dbs_rows_apart(p.heads, oh, tokens, ot, head_dim)) return DBS_ERR_INVALID_ARG;
    from[i] = {(__int128)(uintptr_t)p.x, tokens, xt * xs, p.heads, xh * xs, head_dim * xs};
    to[i] = {(__int128)(uintptr_t)p.out, tokens, ot * os, p.heads, oh * os, head_dim * os};
    const bool in_place = p.x == p.out && x_dtype == out_dtype && (tokens < 2 || xt == ot) && (p.heads < 2 || xh == oh);
    if (!in_place && dbs_rows_meet(from[i], to[i])) return DBS_ERR_INVALID_ARG;
  }
  for (int i = 0; i < count; ++i) {
    if (parts[i].heads == 0) continue;
    const dbs_rows written = to[i].span();
    const void *const at = (const void *)(uintptr_t)written.at;
    const int64_t bytes = (int64_t)written.width;
    if (dbs_overlap(pos, (int64_t)tokens * 4, at, bytes) || dbs_overlap(freq, (int64_t)rot_dim * 4, at, bytes)) return DBS_ERR_INVALID_ARG;
    for (int j = 0; j < count; ++j) {
      if (parts[j].heads == 0) continue;
      if (parts[j].weight && dbs_overlap(parts[j].weight, weight_bytes, at, bytes)) return DBS_ERR_INVALID_ARG;
      if (i != j && (parts_meet(to[i], from[j]) || (i < j && parts_meet(to[i], to[j])))) return DBS_ERR_INVALID_ARG;
    }
  }
  norm_args n = {};
  n.tokens = tokens;
  n.heads = (int)heads;
  n.first_heads = parts[0].heads;
  n.head_dim = head_dim;
  n.rot_dim = rot_dim;
  n.weight_bf16 = weight_dtype == DBS_BF16;
  n.pos = pos;
  n.freq = freq;
  n.scale = scale;
  n.eps = eps;
  for (int i = 0; i < count; ++i)
    n.part[i] = {parts[i].x, parts[i].x_token_stride, parts[i].x_head_stride, parts[i].out, parts[i].out_token_stride,
                 parts[i].out_head_stride, parts[i].weight};
  const bool fx = x_dtype == DBS_F32, fy = out_dtype == DBS_F32;
  const auto run = fx ? (fy ? launch_norm<float, float> : launch_norm<float, bf16_bits>)
                      : (fy ? launch_norm<bf16_bits, float> : launch_norm<bf16_bits, bf16_bits>);
  return run(n, layout == DBS_ROPE_INTERLEAVED, (hipStream_t)stream);
}
