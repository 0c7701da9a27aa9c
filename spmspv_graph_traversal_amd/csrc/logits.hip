// Penalties, biases and masks on rows of logits (dbs_logits_adjust).
#include "values.h"

namespace {

// read in place of an absent list's pointers or an absent row value
__device__ const uint32_t kNothing = 0u;

template <class T>
DBS_DEV T or_nothing(const T *p, int64_t i) {
  typedef const T __attribute__((address_space(1))) *global;
  const global g = p ? (global)(p + i) : (global)(const T *)&kNothing;
  return *g;
}

// Four neighbours, at any alignment of their type.  A vector type: from an array the compiler makes four accesses, of which it
// joins those that the cut case below does not share.
template <class T>
struct four {
  typedef T type __attribute__((ext_vector_type(4)));
  typedef T at_any __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  type v;
  DBS_DEV void load(const T *p, int count) {
    if (count >= 4) v = *(const at_any *)p;
    else
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < count) v[e] = p[e];
  }
  // past the caches: 96 rows of 131072 fp32 logits 25.2 us against 30.7
  DBS_DEV void store(T *p, int count) const {
    if (count >= 4) __builtin_nontemporal_store(v, (at_any *)p);
    else
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < count) p[e] = v[e];
  }
};

// The entries [lo, hi) of a list by all threads, four neighbours to a load; the first AHEAD rounds' loads come before
// whatever stands between fetch() and each().
template <int AHEAD>
struct id_list {
  const int32_t *list;
  int64_t lo, hi;
  four<int32_t> v[AHEAD];

  // row b's part, 0 <= lo <= hi <= len whatever the pointers hold: left() counts on it
  DBS_DEV id_list(const int32_t *ids, const int32_t *ptr, int64_t len, int64_t b) : list(ids) {
    const int32_t first = or_nothing(ptr, b), end = or_nothing(ptr, b + 1);
    lo = first < 0 ? 0 : first > len ? len : first;
    hi = end < lo ? lo : end > len ? len : end;
  }
  DBS_DEV int64_t at(int round) const { return lo + 4 * ((int64_t)round * blockDim.x + threadIdx.x); }
  DBS_DEV int left(int64_t i) const { return (int)(hi - i < 4 ? hi - i : 4); }
  DBS_DEV void fetch() {
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) v[r].load(list + at(r), left(at(r)));
  }
  template <class F>
  DBS_DEV void each(F use) const {
    auto round = [&](const four<int32_t> &ids, int64_t i) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < hi) use(i + e, ids.v[e]);
    };
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) round(v[r], at(r));
    for (int r = AHEAD; at(r) < hi; ++r) {
      four<int32_t> ids;
      ids.load(list + at(r), left(at(r)));
      round(ids, at(r));
    }
  }
};

/*
 * One workgroup per row and slab of the vocabulary, four neighbouring tokens to a thread PIECES times.
 *
 * The history is sparse and unordered, so each workgroup counts the ids that fall into its slab in LDS (integers: any
 * order gives the same counts) instead of in an array in memory that would have to be cleared, filled and read again
 * in every call.  A word holds twice the count of the generated entries, and an odd word or a count means that the id was
 * seen.  The bias of an id that comes twice is its last entry's: the slab keeps the highest entry number.
 *
 * Bound by memory, if a workgroup's chain of loads is kept short: first the logits or, with a mask, its words (logits that
 * it closes are not read at all), the row's scalars at once, the lists, and only then the counting.  96 rows of 131072 fp32
 * logits with 4000 ids, 100 biases and a mask each 24.8 us (114 MB moved, 4.6 TB/s; without lists and mask 20.2, a library
 * copy of the same rows 20.9); one row of 65536 4.2 us, of which the launch is 1.95.  Rows before slabs in the grid, so that
 * a row's lists stay on one die, was slower: 33.7 us against 30.8 (both before the stores past the caches).
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
  auto fetch_logits = [&]() {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int i = 4 * (p * (int)blockDim.x + (int)threadIdx.x);
      in[p].v = 0;
      if (open[p]) in[p].load(logits + b * ld_in + base + i, width - i);
    }
  };
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    const int i = 4 * (p * (int)blockDim.x + (int)threadIdx.x);
    open[p] = i < width ? 15u : 0u;
    if (q.mask && i < width) open[p] = q.mask[b * q.ldmask + ((base + i) >> 5)] >> ((base + i) & 31) & 15u;
  }
  if (!q.mask) fetch_logits();
  id_list<2> hist(q.hist, q.hist_ptr, q.hist_len, b);
  id_list<1> bias(q.bias_idx, q.bias_ptr, q.bias_len, b);
  const int64_t fresh = hist.lo + or_nothing(q.hist_new, b);
  const float rep = or_nothing(q.repetition, b);
  const float freq = or_nothing(q.frequency, b), pres = or_nothing(q.presence, b);
  hist.fetch();
  bias.fetch();
  if (q.hist_ptr || q.bias_ptr) {
    const int words = (q.hist_ptr ? slab : 0) + (q.bias_ptr ? slab : 0);
    for (int i = threadIdx.x; i < words / 4; i += blockDim.x) lds[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (q.mask) fetch_logits();
  dbs_barrier_lds();
  hist.each([&](int64_t at, int32_t id) {
    const uint32_t v = (uint32_t)id - (uint32_t)base;
    if (v < (uint32_t)width) {
      if (at >= fresh) atomicAdd(&count[v], 2u);
      else atomicOr(&count[v], 1u);
    }
  });
  bias.each([&](int64_t at, int32_t id) {
    const uint32_t v = (uint32_t)id - (uint32_t)base;
    if (v < (uint32_t)width) atomicMax(&entry[v], (uint32_t)(at - bias.lo) + 1u);
  });
  dbs_barrier_lds();

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
      const X raw = in[p].v[t];
      float l = dbs_value<X>::load(&raw);
      if (c[t]) {
        if (q.repetition) l = l > 0.0f ? l / rep : l * rep;
        if (c[t] > 1u) l -= freq * (float)(c[t] >> 1) + pres;
      }
      if (e[t]) l += q.bias_val[bias.lo + e[t] - 1];
      if (!(open[p] >> t & 1u)) l = -__builtin_inff();
      o.v[t] = dbs_value<Y>::of(l);
    }
    o.store(out + b * ld_out + base + i, width - i);
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
  // one workgroup of a row writes while others still read that row's lists
  const int64_t written = ((int64_t)(rows - 1) * ld_out + vocab) * dbs_vector_size(out_dtype);
  const auto meets = [&](const void *p, int64_t bytes) { return p && dbs_overlap(p, bytes, out, written); };
  if (meets(q.hist_ptr, ((int64_t)rows + 1) * 4) || meets(q.hist, q.hist_len * 4) || meets(q.hist_new, (int64_t)rows * 4) ||
      meets(q.repetition, (int64_t)rows * 4) || meets(q.frequency, (int64_t)rows * 4) || meets(q.presence, (int64_t)rows * 4) ||
      meets(q.bias_ptr, ((int64_t)rows + 1) * 4) || meets(q.bias_idx, q.bias_len * 4) || meets(q.bias_val, q.bias_len * 4) ||
      meets(q.mask, ((rows - 1) * q.ldmask + ((int64_t)vocab + 31) / 32) * 4))
    return DBS_ERR_INVALID_ARG;
  const bool fx = in_dtype == DBS_F32, fy = out_dtype == DBS_F32;
  auto run = fx ? (fy ? launch_logits<float, float> : launch_logits<float, bf16_bits>)
                : (fy ? launch_logits<bf16_bits, float> : launch_logits<bf16_bits, bf16_bits>);
  return run(rows, vocab, logits, ld_in, q, out, ld_out, (hipStream_t)stream);
}
