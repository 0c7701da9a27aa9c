// Penalties, biases and masks on rows of logits (dbs_logits_adjust).
#include "values.h"

namespace {

// the part [lo, hi) of list `b`, clamped to the list's length
DBS_DEV void list_range(const int32_t *ptr, int64_t len, int64_t b, int64_t &lo, int64_t &hi) {
  lo = ptr[b] < 0 ? 0 : ptr[b];
  hi = ptr[b + 1] > len ? len : ptr[b + 1];
}

// calls use(position, id) for the list's entries [lo, hi), four to a load
template <class F>
DBS_DEV void each_id(const int32_t *list, int64_t lo, int64_t hi, F use) {
  const int64_t step = 4 * blockDim.x;
  int64_t i = lo + 4 * threadIdx.x;
  for (; i + 4 <= hi; i += step) {
    int32_t v[4];
    __builtin_memcpy(v, list + i, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) use(i + e, v[e]);
  }
  for (; i < hi; ++i) use(i, list[i]);  // of one thread: the list's last one to three
}

template <class T>
struct four {
  T v[4];
};
// entries [0, count) of four values at p
template <class T>
DBS_DEV four<T> load_four(const T *p, int count) {
  four<T> f = {};
  if (count >= 4) __builtin_memcpy(&f, p, sizeof f);
  else
    for (int e = 0; e < count; ++e) f.v[e] = p[e];
  return f;
}
template <class T>
DBS_DEV void store_four(T *p, const four<T> &f, int count) {
  if (count >= 4) __builtin_memcpy(p, &f, sizeof f);
  else
    for (int e = 0; e < count; ++e) p[e] = f.v[e];
}

/*
 * One workgroup per row and slab of the vocabulary, four neighbouring tokens to a thread PIECES times.
 *
 * The history is sparse and unordered, so each workgroup counts the ids that fall into its slab in LDS (integers: any
 * order gives the same counts) instead of in an array in memory that would have to be cleared, filled and read again
 * in every call.  A word holds twice the count of the generated entries, and an odd word or a count means that the id was
 * seen.  The bias of an id that comes twice is its last entry's: the slab keeps the highest entry number.
 *
 * Bound by memory: logits read and written once; the lists come from L2 for every slab.  The logits are loaded before the
 * lists are gone through, so that their way from memory is no wait; those that a mask closes are not read at all.
 */
template <class X, class Y, int PIECES>
__global__ __launch_bounds__(512) void k_logits(int vocab, const X *logits, int64_t ld_in, dbs_logits_params q, Y *out,
                                                int64_t ld_out) {
  extern __shared__ uint4 lds[];
  const int64_t b = blockIdx.y;
  const int slab = PIECES * 4 * blockDim.x;
  const int base = blockIdx.x * slab, width = min(slab, vocab - base);
  uint32_t *count = (uint32_t *)lds, *entry = count + (q.hist_ptr ? slab : 0);
  uint32_t open[PIECES];  // a bit for each token of a piece
  four<X> in[PIECES];
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    const int i = 4 * (p * (int)blockDim.x + (int)threadIdx.x);
    open[p] = 15u;
    if (q.mask && i < width) open[p] = q.mask[b * q.ldmask + ((base + i) >> 5)] >> ((base + i) & 31) & 15u;
  }
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    const int i = 4 * (p * (int)blockDim.x + (int)threadIdx.x);
    in[p] = {};
    if (open[p] && i < width) in[p] = load_four(logits + b * ld_in + base + i, width - i);
  }

  int64_t blo = 0;
  if (q.hist_ptr || q.bias_ptr) {
    const int words = (q.hist_ptr ? slab : 0) + (q.bias_ptr ? slab : 0);
    for (int i = threadIdx.x; i < words / 4; i += blockDim.x) lds[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    if (q.hist_ptr) {
      int64_t lo, hi;
      list_range(q.hist_ptr, q.hist_len, b, lo, hi);
      const int64_t fresh = lo + (q.hist_new ? q.hist_new[b] : 0);
      each_id(q.hist, lo, hi, [&](int64_t at, int32_t id) {
        const uint32_t v = (uint32_t)id - (uint32_t)base;
        if (v < (uint32_t)width) {
          if (at >= fresh) atomicAdd(&count[v], 2u);
          else atomicOr(&count[v], 1u);
        }
      });
    }
    if (q.bias_ptr) {
      int64_t hi;
      list_range(q.bias_ptr, q.bias_len, b, blo, hi);
      each_id(q.bias_idx, blo, hi, [&](int64_t at, int32_t id) {
        const uint32_t v = (uint32_t)id - (uint32_t)base;
        if (v < (uint32_t)width) atomicMax(&entry[v], (uint32_t)(at - blo) + 1u);
      });
    }
    __syncthreads();
  }

  const float rep = q.repetition ? q.repetition[b] : 1.0f;
  const float freq = q.frequency ? q.frequency[b] : 0.0f, pres = q.presence ? q.presence[b] : 0.0f;
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    const int at = p * (int)blockDim.x + (int)threadIdx.x, i = 4 * at;
    if (i >= width) continue;
    uint32_t c[4] = {0u, 0u, 0u, 0u}, e[4] = {0u, 0u, 0u, 0u};
    if (q.hist_ptr) __builtin_memcpy(c, (const uint4 *)count + at, 16);
    if (q.bias_ptr) __builtin_memcpy(e, (const uint4 *)entry + at, 16);
    four<Y> o;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      float l = dbs_value<X>::load(&in[p].v[t]);
      if (c[t]) {
        if (q.repetition) l = l > 0.0f ? l / rep : l * rep;
        if (c[t] > 1u) l -= freq * (float)(c[t] >> 1) + pres;
      }
      if (e[t]) l += q.bias_val[blo + e[t] - 1];
      if (!(open[p] >> t & 1u)) l = -__builtin_inff();
      o.v[t] = dbs_value<Y>::of(l);
    }
    store_four(out + b * ld_out + base + i, o, width - i);
  }
}

template <class X, class Y>
dbs_status launch_logits(int rows, int vocab, const void *logits, int64_t ld_in, const dbs_logits_params &q, void *out,
                         int64_t ld_out, hipStream_t s) {
  // Slabs of 4096 tokens: fewer read the lists.  Where they leave compute units idle, slabs of 1024.
  const bool small = (int64_t)rows * ((vocab + 4095ll) / 4096) < 512;
  const int threads = small ? 256 : 512, slab = small ? 1024 : 4096;
  const size_t lds = (size_t)((q.hist_ptr != nullptr) + (q.bias_ptr != nullptr)) * slab * 4;
  const dim3 grid((unsigned)(((int64_t)vocab + slab - 1) / slab), (unsigned)rows);
  const auto kernel = small ? k_logits<X, Y, 1> : k_logits<X, Y, 2>;
  hipLaunchKernelGGL(kernel, grid, dim3(threads), lds, s, vocab, (const X *)logits, ld_in, q, (Y *)out, ld_out);
  return DBS_NOTE(hipGetLastError()) == hipSuccess ? DBS_OK : DBS_ERR_DEVICE;
}

}  // namespace

extern "C" dbs_status dbs_logits_adjust(int32_t rows, int32_t vocab, const void *logits, dbs_dtype in_dtype, int64_t ld_in,
                                        const dbs_logits_params *params, void *out, dbs_dtype out_dtype, int64_t ld_out,
                                        void *stream) {
  if (rows < 0 || vocab < 1 || !params || !dbs_is_vector_dtype(in_dtype) || !dbs_is_vector_dtype(out_dtype))
    return DBS_ERR_INVALID_ARG;
  if (rows > DBS_LOGITS_MAX_ROWS) return DBS_ERR_UNSUPPORTED;
  const dbs_logits_params &q = *params;
  if ((q.hist_ptr != nullptr) != (q.hist != nullptr) && !(q.hist_ptr && q.hist_len == 0)) return DBS_ERR_INVALID_ARG;
  if (!q.hist_ptr && (q.repetition || q.frequency || q.presence || q.hist_new)) return DBS_ERR_INVALID_ARG;
  if (q.bias_ptr ? (q.bias_len > 0 && (!q.bias_idx || !q.bias_val)) : (q.bias_idx || q.bias_val))
    return DBS_ERR_INVALID_ARG;
  if (q.hist_len < 0 || q.bias_len < 0 || q.hist_len >= (int64_t)1 << 31 || q.bias_len >= (int64_t)1 << 31)
    return DBS_ERR_INVALID_ARG;
  if (rows == 0) return DBS_OK;
  if (!logits || !out) return DBS_ERR_INVALID_ARG;
  if (rows > 1 && (ld_in < vocab || ld_out < vocab)) return DBS_ERR_INVALID_ARG;
  if (q.mask && rows > 1 && q.ldmask < ((int64_t)vocab + 31) / 32) return DBS_ERR_INVALID_ARG;
  if (logits == out) {
    if (in_dtype != out_dtype || (rows > 1 && ld_in != ld_out)) return DBS_ERR_INVALID_ARG;
  } else if (dbs_overlap(logits, ((rows - 1) * ld_in + vocab) * dbs_vector_size(in_dtype), out,
                         ((rows - 1) * ld_out + vocab) * dbs_vector_size(out_dtype))) {
    return DBS_ERR_INVALID_ARG;
  }
  const bool fx = in_dtype == DBS_F32, fy = out_dtype == DBS_F32;
  auto run = fx ? (fy ? launch_logits<float, float> : launch_logits<float, bf16_bits>)
                : (fy ? launch_logits<bf16_bits, float> : launch_logits<bf16_bits, bf16_bits>);
  return run(rows, vocab, logits, ld_in, q, out, ld_out, (hipStream_t)stream);
}
