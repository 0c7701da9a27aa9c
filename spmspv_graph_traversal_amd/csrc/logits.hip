// Penalties, biases and masks on rows of logits (dbs_logits_adjust).
#include "values.h"

namespace {

constexpr int kSlab = 4096;  // tokens of one workgroup
constexpr uint32_t kSeen = 0x80000000u;

// the part [lo, hi) of list `b`, clamped to the list's length
DBS_DEV void list_range(const int32_t *ptr, int64_t len, int64_t b, int64_t &lo, int64_t &hi) {
  lo = ptr[b] < 0 ? 0 : ptr[b];
  hi = ptr[b + 1] > len ? len : ptr[b + 1];
}

// One workgroup per row and slab of the vocabulary.  The history is sparse
// and unordered, so each workgroup counts the ids that fall into its slab in
// LDS (integer adds: any order gives the same counts) instead of a count
// array in memory that would have to be cleared, filled and read per call.
// The bias of an id that comes twice is its last entry's: the slab keeps the
// highest entry number.
template <class X, class Y>
__global__ __launch_bounds__(256) void k_logits(int vocab, const X *logits, int64_t ld_in, dbs_logits_params q, Y *out,
                                                int64_t ld_out) {
  __shared__ uint32_t count[kSlab], entry[kSlab];
  const int64_t b = blockIdx.y;
  const int base = blockIdx.x * kSlab, width = min(kSlab, vocab - base);
  const bool hist = q.hist_ptr != nullptr, bias = q.bias_ptr != nullptr;
  for (int i = threadIdx.x; i < kSlab; i += blockDim.x) count[i] = entry[i] = 0u;
  __syncthreads();
  int64_t lo, hi;
  if (hist) {
    list_range(q.hist_ptr, q.hist_len, b, lo, hi);
    const int64_t fresh = lo + (q.hist_new ? q.hist_new[b] : 0);
    for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) {
      const uint32_t v = (uint32_t)q.hist[i] - (uint32_t)base;
      if (v < (uint32_t)width) {
        atomicOr(&count[v], kSeen);
        if (i >= fresh) atomicAdd(&count[v], 1u);
      }
    }
  }
  int64_t blo = 0, bhi = 0;
  if (bias) {
    list_range(q.bias_ptr, q.bias_len, b, blo, bhi);
    for (int64_t i = blo + threadIdx.x; i < bhi; i += blockDim.x) {
      const uint32_t v = (uint32_t)q.bias_idx[i] - (uint32_t)base;
      if (v < (uint32_t)width) atomicMax(&entry[v], (uint32_t)(i - blo) + 1u);
    }
  }
  __syncthreads();
  const float rep = q.repetition ? q.repetition[b] : 1.0f;
  const float freq = q.frequency ? q.frequency[b] : 0.0f, pres = q.presence ? q.presence[b] : 0.0f;
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    const int v = base + i;
    float l = -__builtin_inff();
    if (!q.mask || (q.mask[b * q.ldmask + (v >> 5)] >> (v & 31)) & 1u) {
      l = dbs_value<X>::load(logits + b * ld_in + v);
      const uint32_t c = count[i];
      if (c) {
        if (q.repetition) l = l > 0.0f ? l / rep : l * rep;
        const uint32_t fresh = c & ~kSeen;
        if (fresh) l -= freq * (float)fresh + pres;
      }
      if (entry[i]) l += q.bias_val[blo + entry[i] - 1];
    }
    out[b * ld_out + v] = dbs_value<Y>::of(l);
  }
}

template <class X, class Y>
dbs_status launch_logits(int rows, int vocab, const void *logits, int64_t ld_in, const dbs_logits_params &q, void *out,
                         int64_t ld_out, hipStream_t s) {
  const unsigned slabs = ((unsigned)vocab + kSlab - 1) / kSlab;
  hipLaunchKernelGGL((k_logits<X, Y>), dim3(slabs, (unsigned)rows), dim3(256), 0, s, vocab, (const X *)logits, ld_in, q,
                     (Y *)out, ld_out);
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
