// Loads and stores of the fp32 and bf16 vectors of the decode-step operators.
#pragma once

#include "common.h"

typedef unsigned short bf16_bits;

template <class T>
struct dbs_value;
template <>
struct dbs_value<float> {
  static constexpr dbs_dtype dtype = DBS_F32;
  DBS_DEV static float load(const float *p) { return *p; }
  DBS_DEV static float of(float v) { return v; }
};
template <>
struct dbs_value<bf16_bits> {
  static constexpr dbs_dtype dtype = DBS_BF16;
  DBS_DEV static float load(const bf16_bits *p) { return bf16_to_f32(*p); }
  // round to nearest, ties to even; a NaN keeps its sign and becomes quiet
  DBS_DEV static bf16_bits of(float v) {
    const uint32_t u = __float_as_uint(v);
    if (v != v) return (bf16_bits)((u >> 16) | 0x40u);
    return (bf16_bits)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
  }
};

inline bool dbs_is_vector_dtype(int dtype) { return dtype == DBS_F32 || dtype == DBS_BF16; }
inline int64_t dbs_vector_size(int dtype) { return dtype == DBS_F32 ? 4 : 2; }

// whether [a, a + abytes) and [b, b + bbytes) share a byte
inline bool dbs_overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
  const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
  return abytes > 0 && bbytes > 0 && p < q + (uintptr_t)bbytes && q < p + (uintptr_t)abytes;
}

// a barrier that waits for LDS only, not for loads from memory in flight
DBS_DEV void dbs_barrier_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
