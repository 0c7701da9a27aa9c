// Rotary positions (dbs_rope) and their frequencies (dbs_rope_frequencies).
#include <math.h>

#include "values.h"

namespace {

// One workgroup per token.  Its cosines and sines are computed once, in 64
// bits up to the fraction of a turn (a position times a frequency is many
// turns; 32 bits would lose its phase), and used by every head.
template <class X, class Y>
__global__ __launch_bounds__(256) void k_rope(int heads, int head_dim, int rot_dim, int interleaved,
                                              const int32_t *__restrict__ pos, const double *__restrict__ freq,
                                              float scale, float direction, const X *x, int64_t xt, int64_t xh,
                                              Y *out, int64_t ot, int64_t oh) {
  __shared__ float2 turn[DBS_ROPE_MAX_DIM / 2];
  const int64_t t = blockIdx.x;
  const int p = pos[t];
  if (p < 0) return;
  const int half = rot_dim / 2;
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const double turns = (double)p * freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    turn[i] = make_float2(scale * c, scale * direction * s);
  }
  __syncthreads();
  const X *xb = x + t * xt;
  Y *ob = out + t * ot;
  const int units = half + (head_dim - rot_dim);  // pairs, then copied elements
  const int64_t total = (int64_t)heads * units;
  for (int64_t u = threadIdx.x; u < total; u += blockDim.x) {
    const int h = (int)(u / units), i = (int)(u % units);
    const X *xp = xb + h * xh;
    Y *op = ob + h * oh;
    if (i < half) {
      const int ia = interleaved ? 2 * i : i, ib = interleaved ? 2 * i + 1 : i + half;
      const float a = dbs_value<X>::load(xp + ia), b = dbs_value<X>::load(xp + ib);
      const float2 w = turn[i];
      op[ia] = dbs_value<Y>::of(a * w.x - b * w.y);
      op[ib] = dbs_value<Y>::of(a * w.y + b * w.x);
    } else {
      const int d = rot_dim + (i - half);
      op[d] = dbs_value<Y>::of(dbs_value<X>::load(xp + d));
    }
  }
}

template <class X, class Y>
dbs_status launch_rope(int tokens, int heads, int head_dim, int rot_dim, int layout, const int32_t *pos,
                       const double *freq, float scale, int inverse, const void *x, int64_t xt, int64_t xh, void *out,
                       int64_t ot, int64_t oh, hipStream_t s) {
  hipLaunchKernelGGL((k_rope<X, Y>), dim3((unsigned)tokens), dim3(256), 0, s, heads, head_dim, rot_dim,
                     layout == DBS_ROPE_INTERLEAVED, pos, freq, scale, inverse ? -1.0f : 1.0f, (const X *)x, xt, xh,
                     (Y *)out, ot, oh);
  return DBS_NOTE(hipGetLastError()) == hipSuccess ? DBS_OK : DBS_ERR_DEVICE;
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
  if (rot_dim > DBS_ROPE_MAX_DIM) return DBS_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0) return DBS_OK;
  if (!pos || (rot_dim > 0 && !freq) || !x || !out) return DBS_ERR_INVALID_ARG;
  // rows of one output may not overlap each other, and an in-place call reads what it writes
  if (heads > 1 && oh < head_dim && oh > -(int64_t)head_dim) return DBS_ERR_INVALID_ARG;
  if (tokens > 1 && ot < head_dim && ot > -(int64_t)head_dim) return DBS_ERR_INVALID_ARG;
  if (x == out && (x_dtype != out_dtype || (tokens > 1 && xt != ot) || (heads > 1 && xh != oh)))
    return DBS_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  const bool fx = x_dtype == DBS_F32, fy = out_dtype == DBS_F32;
  auto run = fx ? (fy ? launch_rope<float, float> : launch_rope<float, bf16_bits>)
                : (fy ? launch_rope<bf16_bits, float> : launch_rope<bf16_bits, bf16_bits>);
  return run(tokens, heads, head_dim, rot_dim, layout, pos, freq, scale, inverse, x, xt, xh, out, ot, oh, s);
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
