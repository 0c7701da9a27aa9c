// Rotary positions (dbs_rope) and their frequencies (dbs_rope_frequencies).
#include <math.h>

#include "values.h"

namespace {

// past the caches: 8192 tokens of 40 heads of 128 bf16 30.6 us against 35.0
template <class T, int W>
DBS_DEV void write(T *p, const T (&v)[W]) {
  typedef T at_any __attribute__((ext_vector_type(W), aligned(sizeof(T))));
  at_any w;
  __builtin_memcpy(&w, v, sizeof v);
  __builtin_nontemporal_store(w, (at_any *)p);
}

/*
 * Mathematics: a pair (a, b) of a head turns by p = position * freq[i].  Cosine and sine depend on the token and the pair
 * alone, so a workgroup computes them once per token into LDS and uses them for its heads.  The turn is formed and reduced in 64
 * bits (a far position is many turns, of which 32 bits would keep no fraction), the sine of its fraction in 32.
 *
 * One workgroup per token and `per` heads, W pairs or W copied elements to a lane at a time, 16 bytes where the sizes allow;
 * W = 1 takes any rot_dim and head_dim.  Bound by memory for a prompt: 8192 tokens of 40 heads of 128 bf16 30.6 us, 168 MB at
 * 5.5 TB/s (interleaved 27.0).  One token takes 2.3 us, the launch being 1.95: x is loaded before the sines, so that its chain
 * is not position, frequencies, sines and then x.
 */
template <class X, class Y, int W, bool INTERLEAVED>
struct rope_unit {
  // Half layout, or W = 1: W pairs, or W elements from rot_dim on.  Interleaved with W > 1: 2 W neighbours, of which those
  // from rot_dim on are copied.
  static constexpr bool kMixed = INTERLEAVED && W > 1;
  X a[W], b[W];
  int h, i;

  DBS_DEV void load(const X *x, int64_t xh, int u, int units, int turned, int half) {
    h = u / units;
    i = u % units;
    const X *p = x + h * xh;
    if (kMixed || i < turned) {
      __builtin_memcpy(a, p + (INTERLEAVED ? 2 * W * i : W * i), sizeof a);
      __builtin_memcpy(b, p + (INTERLEAVED ? 2 * W * i + W : half + W * i), sizeof b);
    } else {
      __builtin_memcpy(a, p + 2 * half + W * (i - turned), sizeof a);
    }
  }
  DBS_DEV void store(Y *out, int64_t oh, const float2 *turn, int turned, int half) const {
    Y oa[W], ob[W];
    Y *p = out + h * oh;
    if (kMixed || i < turned) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const int ka = INTERLEAVED ? 2 * e : e, kb = INTERLEAVED ? 2 * e + 1 : W + e;  // within a, b
        const float va = dbs_value<X>::load(ka < W ? &a[ka % W] : &b[ka % W]);
        const float vb = dbs_value<X>::load(kb < W ? &a[kb % W] : &b[kb % W]);
        float ra = va, rb = vb;
        if (!kMixed || W * i + e < half) {
          const float2 w = turn[W * i + e];
          ra = va * w.x - vb * w.y;
          rb = va * w.y + vb * w.x;
        }
        (ka < W ? oa[ka % W] : ob[ka % W]) = dbs_value<Y>::of(ra);
        (kb < W ? oa[kb % W] : ob[kb % W]) = dbs_value<Y>::of(rb);
      }
      write(p + (INTERLEAVED ? 2 * W * i : W * i), oa);
      write(p + (INTERLEAVED ? 2 * W * i + W : half + W * i), ob);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) oa[e] = dbs_value<Y>::of(dbs_value<X>::load(&a[e]));
      write(p + 2 * half + W * (i - turned), oa);
    }
  }
};

// units of a head
template <int W, bool INTERLEAVED>
__host__ __device__ inline int rope_units(int head_dim, int rot_dim) {
  return INTERLEAVED && W > 1 ? head_dim / (2 * W) : rot_dim / 2 / W + (head_dim - rot_dim) / W;
}

template <class X, class Y, int W, bool INTERLEAVED>
__global__ __launch_bounds__(512) void k_rope(int heads, int per, int head_dim, int rot_dim,
                                              const int32_t *__restrict__ pos, const double *__restrict__ freq,
                                              float scale, float direction, const X *x, int64_t xt, int64_t xh, Y *out,
                                              int64_t ot, int64_t oh) {
  __shared__ float2 turn[DBS_ROPE_MAX_DIM / 2];
  const int64_t t = blockIdx.x;
  const int p = pos[t];
  if (p < 0) return;
  const int half = rot_dim / 2, h0 = blockIdx.y * per, count = min(per, heads - h0);
  x += t * xt + h0 * xh;
  out += t * ot + h0 * oh;
  const int turned = half / W, units = rope_units<W, INTERLEAVED>(head_dim, rot_dim), all = count * units;
  rope_unit<X, Y, W, INTERLEAVED> now;
  int u = threadIdx.x;
  if (u < all) now.load(x, xh, u, units, turned, half);
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const double turns = (double)p * freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    turn[i] = make_float2(scale * c, scale * direction * s);
  }
  dbs_barrier_lds();
  if (u < all) now.store(out, oh, turn, turned, half);
  for (u += blockDim.x; u < all; u += blockDim.x) {
    now.load(x, xh, u, units, turned, half);
    now.store(out, oh, turn, turned, half);
  }
}

struct rope_args {
  int tokens, heads, head_dim, rot_dim;
  bool interleaved;
  const int32_t *pos;
  const double *freq;
  float scale, direction;
  const void *x;
  int64_t xt, xh;
  void *out;
  int64_t ot, oh;
};

template <class X, class Y, int W, bool INTERLEAVED>
dbs_status launch_rope(const rope_args &r, hipStream_t s) {
  // All heads of a token share its sines; few tokens are spread over workgroups of 256 lanes by head, or one would do the
  // work of a chip.
  const int units = rope_units<W, INTERLEAVED>(r.head_dim, r.rot_dim);
  int per = r.heads;
  if (r.tokens < 512) per = units >= 256 ? 1 : 256 / units;
  if (per > r.heads) per = r.heads;
  if (per < (r.heads + 65534) / 65535) per = (r.heads + 65534) / 65535;  // the grid's limit
  // rounds of at most 512 lanes, all nearly full
  const int64_t all = (int64_t)per * units, rounds = (all + 511) / 512;
  const int threads = (int)((all + rounds * 64 - 1) / (rounds * 64)) * 64;
  // a launch's lanes are counted in 32 bits
  const int most = (int)(0x7FFFFFFF / threads);
  for (int t = 0;; t += most) {
    const int count = r.tokens - t < most ? r.tokens - t : most;
    const dim3 grid((unsigned)count, (unsigned)((r.heads + per - 1) / per));
    hipLaunchKernelGGL((k_rope<X, Y, W, INTERLEAVED>), grid, dim3(threads), 0, s, r.heads, per, r.head_dim, r.rot_dim,
                       r.pos + t, r.freq, r.scale, r.direction, (const X *)r.x + t * r.xt, r.xt, r.xh,
                       (Y *)r.out + t * r.ot, r.ot, r.oh);
    if (DBS_NOTE(hipGetLastError()) != hipSuccess) return DBS_ERR_DEVICE;
    if (count == r.tokens - t) return DBS_OK;
  }
}

// The widest units that the sizes are made of, up to 16 bytes a lane: wider ones would leave gaps between the lanes' stores,
// which past the caches cost whole lines (2000 tokens of 32 heads of 256, 64 rotated, bf16 to fp32: 52 us with 64 bytes).
template <class X, class Y>
dbs_status launch_rope(const rope_args &r, hipStream_t s) {
  constexpr int most = 16 / (sizeof(X) > sizeof(Y) ? sizeof(X) : sizeof(Y));
  if (r.interleaved) {
    if (r.head_dim % most == 0) return launch_rope<X, Y, most / 2, true>(r, s);
    if (most == 8 && r.head_dim % 4 == 0) return launch_rope<X, Y, 2, true>(r, s);
    return launch_rope<X, Y, 1, true>(r, s);
  }
  const int width = r.rot_dim / 2 | (r.head_dim - r.rot_dim);
  if (width % most == 0) return launch_rope<X, Y, most, false>(r, s);
  if (most == 8 && width % 4 == 0) return launch_rope<X, Y, 4, false>(r, s);
  if (width % 2 == 0) return launch_rope<X, Y, 2, false>(r, s);
  return launch_rope<X, Y, 1, false>(r, s);
}

// whether rows of `width` elements at i * si + j * sj are disjoint because each i's rows end before the next i's begin
bool apart(int64_t ni, int64_t si, int64_t nj, int64_t sj, int64_t width) {
  typedef __int128 wide;
  const wide i = si < 0 ? -(wide)si : si, j = sj < 0 ? -(wide)sj : sj;
  return (nj < 2 || j >= width) && (ni < 2 || i >= (nj - 1) * j + width);
}

}  // namespace

extern "C" dbs_status dbs_rope(int32_t tokens, int32_t heads, int32_t head_dim, int32_t rot_dim, dbs_rope_layout layout,
                               const int32_t *pos, const double *freq, float scale, int32_t inverse, const void *x,
                               dbs_dtype x_dtype, int64_t xt, int64_t xh, void *out, dbs_dtype out_dtype, int64_t ot,
                               int64_t oh, void *stream) {
  if (tokens < 0 || heads < 0 || head_dim < 1 || rot_dim < 0 || rot_dim > head_dim || (rot_dim & 1))
    return DBS_ERR_INVALID_ARG;
  if (layout != DBS_ROPE_HALF && layout != DBS_ROPE_INTERLEAVED) return DBS_ERR_INVALID_ARG;
  if (!dbs_is_vector_dtype(x_dtype) || !dbs_is_vector_dtype(out_dtype)) return DBS_ERR_INVALID_ARG;
  // a lane's counter passes the number of elements by up to a workgroup's lanes, in 32 bits
  if (rot_dim > DBS_ROPE_MAX_DIM || (int64_t)heads * head_dim > DBS_ROPE_MAX_ELEMENTS) return DBS_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0) return DBS_OK;
  if (!pos || (rot_dim > 0 && !freq) || !x || !out) return DBS_ERR_INVALID_ARG;
  // two heads of the output may not share an element, and an in-place call reads what it writes
  if (!apart(tokens, ot, heads, oh, head_dim) && !apart(heads, oh, tokens, ot, head_dim)) return DBS_ERR_INVALID_ARG;
  const bool in_place = x == out && x_dtype == out_dtype && (tokens < 2 || xt == ot) && (heads < 2 || xh == oh);
  const __int128 xs = dbs_vector_size(x_dtype), os = dbs_vector_size(out_dtype);
  const dbs_rows from = {(__int128)(uintptr_t)x, tokens, xt * xs, heads, xh * xs, head_dim * xs};
  const dbs_rows to = {(__int128)(uintptr_t)out, tokens, ot * os, heads, oh * os, head_dim * os};
  // else workgroups would read what others write
  if (!in_place && dbs_rows_meet(from, to)) return DBS_ERR_INVALID_ARG;
  const dbs_rows written = to.span();
  if (dbs_overlap(pos, (int64_t)tokens * 4, (const void *)(uintptr_t)written.at, (int64_t)written.width) ||
      dbs_overlap(freq, (int64_t)rot_dim * 4, (const void *)(uintptr_t)written.at, (int64_t)written.width))
    return DBS_ERR_INVALID_ARG;
  const rope_args r = {tokens, heads, head_dim, rot_dim, layout == DBS_ROPE_INTERLEAVED, pos, freq, scale,
                       inverse ? -1.0f : 1.0f, x, xt, xh, out, ot, oh};
  const bool fx = x_dtype == DBS_F32, fy = out_dtype == DBS_F32;
  auto run = fx ? (fy ? launch_rope<float, float> : launch_rope<float, bf16_bits>)
                : (fy ? launch_rope<bf16_bits, float> : launch_rope<bf16_bits, bf16_bits>);
  return run(r, (hipStream_t)stream);
}

extern "C" dbs_status dbs_rope_frequencies(const dbs_rope_options *o, double *freq, float *scale) {
  if (!o || !freq || o->rot_dim < 2 || (o->rot_dim & 1) || o->rot_dim > DBS_ROPE_MAX_DIM) return DBS_ERR_INVALID_ARG;
  if (o->scaling < DBS_ROPE_PLAIN || o->scaling > DBS_ROPE_RAMP) return DBS_ERR_INVALID_ARG;
  if (!(o->base > 1.0) || !isfinite(o->base)) return DBS_ERR_INVALID_ARG;
  if (o->scaling != DBS_ROPE_PLAIN && (!(o->factor >= 1.0) || !isfinite(o->factor))) return DBS_ERR_INVALID_ARG;
  const bool banded = o->scaling == DBS_ROPE_BANDS || o->scaling == DBS_ROPE_RAMP;
  if (banded && (!(o->low > 0.0) || !(o->high > o->low) || !isfinite(o->high) || !(o->context > 0.0) ||
                 !isfinite(o->context)))
    return DBS_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586477;
  const int half = o->rot_dim / 2;
  double base = o->base, first = 0.0, last = 0.0;
  if (o->scaling == DBS_ROPE_BASE) {
    if (o->rot_dim == 2) return DBS_ERR_INVALID_ARG;  // its one frequency is 1 whatever the base
    base *= pow(o->factor, (double)o->rot_dim / (o->rot_dim - 2));
  }
  if (o->scaling == DBS_ROPE_RAMP) {
    const double per = o->rot_dim / (2.0 * log(o->base));
    first = fmax(floor(per * log(o->context / (two_pi * o->high))), 0.0);
    last = fmin(ceil(per * log(o->context / (two_pi * o->low))), o->rot_dim - 1.0);
    if (last <= first) last = first + 0.001;  // a step in place of a ramp of no width
  }
  for (int i = 0; i < half; ++i) {
    double f = pow(base, -(double)i / half);
    if (o->scaling == DBS_ROPE_LINEAR) f /= o->factor;
    if (o->scaling == DBS_ROPE_BANDS) {
      const double t = o->context * f / two_pi;
      const double w = fmin(fmax((t - o->low) / (o->high - o->low), 0.0), 1.0);
      f *= (1.0 - w) / o->factor + w;
    }
    if (o->scaling == DBS_ROPE_RAMP) {
      const double w = fmin(fmax((i - first) / (last - first), 0.0), 1.0);
      f *= w / o->factor + (1.0 - w);
    }
    freq[i] = f;
  }
  if (scale) *scale = o->scaling == DBS_ROPE_RAMP ? (float)(0.1 * log(o->factor) + 1.0) : 1.0f;
  return DBS_OK;
}
