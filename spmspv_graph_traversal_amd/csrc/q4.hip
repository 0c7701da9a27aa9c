// Products of a matrix of 4-bit codes with group scales: layout (dbs_q4_build),
// y = W x (dbs_q4_product), with a row mask (dbs_q4_product_masked) and the
// gate and up layers in one pass (dbs_q4_gated).
#include <string.h>

#include <new>

#include "q4_tiles.h"

namespace {

// a code dword of the layout to a thread at a time
__global__ __launch_bounds__(256) void k_q4_codes(int m, int n, int group, int mt, int kt, const uint8_t *__restrict__ codes,
                                                  const uint8_t *__restrict__ zeros, uint32_t *__restrict__ out) {
  const int64_t all = (int64_t)mt * kt * 256, groups = ((int64_t)n + group - 1) / group;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t tile = i >> 8;
    const int lane = (int)(i >> 2) & 63, s = (int)i & 3;
    const int64_t row = tile / kt * Q4_ROWS + (lane & 15);
    const int64_t col0 = tile % kt * Q4_COLS + 32 * s + 8 * (lane >> 4);
    uint32_t w = 0u;
    for (int e = 0; e < 8; ++e) {
      uint32_t c = 8u;
      const int64_t col = col0 + e;
      if (row < m && col < n) {
        const uint8_t two = codes[row * (((int64_t)n + 1) / 2) + (col >> 1)];
        c = (col & 1) ? two >> 4 : two & 15u;
      } else if (row < m && zeros && col / group < groups) {
        c = zeros[row * groups + col / group] & 15u;  // the rest of a cut group: weight zero
      }
      const int b = q4_code_bit(e);
      w |= c << b;
      if (b > 28) w |= c >> (32 - b);
    }
    out[i] = w;
  }
}

// whether all weights of a row's columns [low, high) are zero: low even, `row` the row's codes
DBS_DEV bool q4_all_zero(const uint8_t *row, int64_t low, int64_t high, uint32_t zero) {
  for (int64_t c = low; c < high; c += 2)
    if ((row[c >> 1] ^ zero * 17u) & (c + 1 < high ? 255u : 15u)) return false;
  return true;
}

// A record to a thread at a time; a zero point above 15 sets *bad.  A group whose weights are all zero gets the scale 0: the
// products subtract sums of (16 + zero) x from sums of (16 + code) x that are rounded apart, and would leave some 2^-24 of these.
// (An infinite or NaN scale stays, its weights are NaN.)
template <class S>
__global__ __launch_bounds__(256) void k_q4_records(int m, int n, int group, int mt, int kt, const uint8_t *__restrict__ codes,
                                                    const S *__restrict__ scales, const uint8_t *__restrict__ zeros,
                                                    uint32_t *__restrict__ out, uint32_t *bad) {
  const int gpt = Q4_COLS / group;
  const int64_t all = (int64_t)mt * kt * Q4_ROWS * gpt, groups = ((int64_t)n + group - 1) / group;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t tile = i / (Q4_ROWS * gpt);
    const int64_t row = tile / kt * Q4_ROWS + (i / gpt) % Q4_ROWS, g = tile % kt * gpt + i % gpt;
    const bool in = row < m && g < groups;
    uint32_t z = 8u;
    if (in && zeros) z = zeros[row * groups + g];
    if (z > 15u) *bad = 1u;
    const float off = (float)(16u + z);
    uint32_t scale = 0u;  // as fp32
    if (in) {
      scale = sizeof(S) == 4 ? __float_as_uint((float)scales[row * groups + g]) : (uint32_t)scales[row * groups + g] << 16;
      const int64_t low = g * group, high = low + group < n ? low + group : n;
      if ((scale & 0x7F800000u) != 0x7F800000u && q4_all_zero(codes + row * (((int64_t)n + 1) / 2), low, high, z)) scale = 0u;
    }
    if (sizeof(S) == 4) {
      out[2 * i] = scale;
      out[2 * i + 1] = __float_as_uint(off);
    } else {
      out[i] = scale | __float_as_uint(off) >> 16;
    }
  }
}

// checks shared by the products, then the launch
dbs_status product(dbs_q4_handle A, dbs_q4_handle U, int act, int32_t tokens, const void *x, dbs_dtype xd, int64_t ldx,
                   const uint32_t *mask, int64_t ldmask, float fill, void *y, dbs_dtype yd, int64_t ldy, void *stream) {
  if (!A || tokens < 0 || !dbs_is_vector_dtype(xd) || !dbs_is_vector_dtype(yd)) return DBS_ERR_INVALID_ARG;
  if (tokens > DBS_Q4_MAX_TOKENS) return DBS_ERR_UNSUPPORTED;
  int dev = -1;
  if (DBS_NOTE(hipGetDevice(&dev)) != hipSuccess) return DBS_ERR_DEVICE;
  if (dev != A->device) return DBS_ERR_INVALID_ARG;
  if (U && (U->device != dev || U->m != A->m || U->n != A->n || U->group != A->group || U->scale_dtype != A->scale_dtype))
    return DBS_ERR_INVALID_ARG;
  if (tokens == 0) return DBS_OK;
  if (!x || !y) return DBS_ERR_INVALID_ARG;
  if (tokens > 1 && (ldx < A->n || ldy < A->m || (mask && ldmask < ((int64_t)A->m + 31) / 32))) return DBS_ERR_INVALID_ARG;
  const int64_t last = tokens - 1;
  const int64_t ybytes = (last * ldy + A->m) * dbs_vector_size(yd);
  if (dbs_overlap(x, (last * ldx + A->n) * dbs_vector_size(xd), y, ybytes)) return DBS_ERR_INVALID_ARG;
  if (mask && dbs_overlap(mask, (last * ldmask + ((int64_t)A->m + 31) / 32) * 4, y, ybytes)) return DBS_ERR_INVALID_ARG;
  q4_args q = {dev, {A->codes, U ? U->codes : nullptr}, {A->recs, U ? U->recs : nullptr}, A->m, A->n, A->mt, A->kt, act,
               tokens, x, ldx, mask, ldmask, fill, yd == DBS_BF16, y, ldy};
  const auto run = xd == DBS_BF16 ? (U ? dbs_q4_launch_bf16_gated : dbs_q4_launch_bf16)
                                  : (U ? dbs_q4_launch_f32_gated : dbs_q4_launch_f32);
  const q4_shape shape = q4_pick_shape(A->mt, A->kt, tokens, xd, U != nullptr, mask != nullptr);
  const hipError_t e = run(q, q4_record_words(A->scale_dtype), A->gpt, shape, (hipStream_t)stream);
  return e == hipSuccess ? DBS_OK : DBS_ERR_DEVICE;
}

void q4_free(dbs_q4_matrix *A) {
  if (A->codes) (void)hipFree(A->codes);
  if (A->recs) (void)hipFree(A->recs);
  delete A;
}

dbs_status map_err(hipError_t e) {
  if (e == hipSuccess) return DBS_OK;
  (void)hipGetLastError();
  return e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation ? DBS_ERR_OUT_OF_MEMORY : DBS_ERR_DEVICE;
}

dbs_status q4_build(dbs_q4_matrix *A, const uint8_t *codes, const void *scales, const uint8_t *zeros, hipStream_t s) {
  const int64_t tiles = (int64_t)A->mt * A->kt;
  const int64_t nrec = tiles * Q4_ROWS * A->gpt;
  const int64_t code_bytes = tiles * Q4_TILE_BYTES, rec_bytes = nrec * 4 * q4_record_words(A->scale_dtype);
  hipError_t e;
  // the check flag behind the records
  if ((e = DBS_NOTE(hipMalloc((void **)&A->codes, (size_t)code_bytes))) != hipSuccess) return map_err(e);
  if ((e = DBS_NOTE(hipMalloc((void **)&A->recs, (size_t)rec_bytes + 4))) != hipSuccess) return map_err(e);
  A->bytes = code_bytes + rec_bytes + 4;
  uint32_t *bad = A->recs + rec_bytes / 4;
  if ((e = DBS_NOTE(hipMemsetAsync(bad, 0, 4, s))) != hipSuccess) return map_err(e);
  // a launch's lanes are counted in 32 bits, a large matrix's dwords are not
  const int64_t most = 16384, g1 = tiles < most ? tiles : most, g2 = (nrec + 255) / 256 < most ? (nrec + 255) / 256 : most;
  hipLaunchKernelGGL(k_q4_codes, dim3((unsigned)g1), dim3(256), 0, s, A->m, A->n, A->group, A->mt, A->kt, codes, zeros, A->codes);
  if (A->scale_dtype == DBS_F32)
    hipLaunchKernelGGL(k_q4_records<float>, dim3((unsigned)g2), dim3(256), 0, s, A->m, A->n, A->group, A->mt, A->kt, codes,
                       (const float *)scales, zeros, A->recs, bad);
  else
    hipLaunchKernelGGL(k_q4_records<bf16_bits>, dim3((unsigned)g2), dim3(256), 0, s, A->m, A->n, A->group, A->mt, A->kt, codes,
                       (const bf16_bits *)scales, zeros, A->recs, bad);
  if ((e = DBS_NOTE(hipGetLastError())) != hipSuccess) return map_err(e);
  uint32_t h = 0;
  if ((e = DBS_NOTE(hipMemcpyAsync(&h, bad, 4, hipMemcpyDeviceToHost, s))) != hipSuccess) return map_err(e);
  if ((e = DBS_NOTE(hipStreamSynchronize(s))) != hipSuccess) return map_err(e);
  return h ? DBS_ERR_INVALID_ARG : DBS_OK;
}

}  // namespace

extern "C" {

dbs_status dbs_q4_build(int32_t m, int32_t n, int32_t group, const uint8_t *codes, const void *scales,
                        dbs_dtype scale_dtype, const uint8_t *zeros, void *stream, dbs_q4_handle *out) {
  if (!out || m < 1 || n < 1 || !codes || !scales || !dbs_is_vector_dtype(scale_dtype)) return DBS_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return DBS_ERR_INVALID_ARG;
  if (m > DBS_Q4_MAX_ROWS || n > DBS_Q4_MAX_COLUMNS) return DBS_ERR_UNSUPPORTED;
  dbs_q4_matrix *A = new (std::nothrow) dbs_q4_matrix;
  if (!A) return DBS_ERR_OUT_OF_MEMORY;
  memset((void *)A, 0, sizeof(*A));
  A->m = m;
  A->n = n;
  A->group = group;
  A->scale_dtype = scale_dtype;
  A->mt = (int32_t)(((int64_t)m + Q4_ROWS - 1) / Q4_ROWS);
  A->kt = (int32_t)(((int64_t)n + Q4_COLS - 1) / Q4_COLS);
  A->gpt = Q4_COLS / group;
  dbs_status st = map_err(DBS_NOTE(hipGetDevice(&A->device)));
  if (st == DBS_OK) st = q4_build(A, codes, scales, zeros, (hipStream_t)stream);
  if (st != DBS_OK) {
    q4_free(A);
    return st;
  }
  *out = A;
  return DBS_OK;
}

dbs_status dbs_q4_bytes(dbs_q4_handle A, int64_t *bytes) {
  if (!A || !bytes) return DBS_ERR_INVALID_ARG;
  *bytes = A->bytes;
  return DBS_OK;
}

dbs_status dbs_q4_free(dbs_q4_handle A) {
  if (A) q4_free(A);
  return DBS_OK;
}

dbs_status dbs_q4_product(dbs_q4_handle A, int32_t tokens, const void *x, dbs_dtype x_dtype, int64_t ldx, void *y,
                          dbs_dtype y_dtype, int64_t ldy, void *stream) {
  return product(A, nullptr, 0, tokens, x, x_dtype, ldx, nullptr, 0, 0.0f, y, y_dtype, ldy, stream);
}

dbs_status dbs_q4_product_masked(dbs_q4_handle A, int32_t tokens, const void *x, dbs_dtype x_dtype, int64_t ldx,
                                 const uint32_t *row_mask, int64_t ldmask, float fill, void *y, dbs_dtype y_dtype,
                                 int64_t ldy, void *stream) {
  if (!row_mask && tokens != 0) return DBS_ERR_INVALID_ARG;
  return product(A, nullptr, 0, tokens, x, x_dtype, ldx, row_mask, ldmask, fill, y, y_dtype, ldy, stream);
}

dbs_status dbs_q4_gated(dbs_q4_handle G, dbs_q4_handle U, dbs_activation act, int32_t tokens, const void *x,
                        dbs_dtype x_dtype, int64_t ldx, void *y, dbs_dtype y_dtype, int64_t ldy, void *stream) {
  if (!U || (act != DBS_ACT_SILU && act != DBS_ACT_GELU_TANH && act != DBS_ACT_RELU)) return DBS_ERR_INVALID_ARG;
  return product(G, U, act, tokens, x, x_dtype, ldx, nullptr, 0, 0.0f, y, y_dtype, ldy, stream);
}

}  // extern "C"
