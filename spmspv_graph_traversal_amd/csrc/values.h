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

// Values rounded to the type, to nearest with ties to even, two bf16 to an instruction (dbs_value::of takes six for one).
template <int W>
DBS_DEV void dbs_round(float (&to)[W], const float (&v)[W]) {
#pragma unroll
  for (int e = 0; e < W; ++e) to[e] = v[e];
}
template <int W>
DBS_DEV void dbs_round(bf16_bits (&to)[W], const float (&v)[W]) {
  typedef float wide __attribute__((ext_vector_type(W)));
  typedef __bf16 narrow __attribute__((ext_vector_type(W)));
  wide w;
  __builtin_memcpy(&w, v, sizeof v);
  const narrow n = __builtin_convertvector(w, narrow);
  __builtin_memcpy(to, &n, sizeof to);
}

inline bool dbs_is_vector_dtype(int dtype) { return dtype == DBS_F32 || dtype == DBS_BF16; }
inline int64_t dbs_vector_size(int dtype) { return dtype == DBS_F32 ? 4 : 2; }

// whether [a, a + abytes) and [b, b + bbytes) share a byte
inline bool dbs_overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
  const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
  return abytes > 0 && bbytes > 0 && p < q + (uintptr_t)bbytes && q < p + (uintptr_t)abytes;
}

// Rows of `width` bytes at `at` + i * si + j * sj, i below ni and j below nj (si and sj of any sign, in bytes).
struct dbs_rows {
  __int128 at, ni, si, nj, sj, width;
  // the bytes from the first to behind the last one, as one row
  dbs_rows span() const {
    const __int128 li = (ni - 1) * si, lj = (nj - 1) * sj;
    const __int128 low = (li < 0 ? li : 0) + (lj < 0 ? lj : 0), high = (li > 0 ? li : 0) + (lj > 0 ? lj : 0) + width;
    return {at + low, 1, 0, 1, 0, high - low};
  }
  dbs_rows turned() const { return {at, nj, sj, ni, si, width}; }
  // of one i each: all its j as one row
  dbs_rows joined() const {
    const dbs_rows all = dbs_rows{at, 1, 0, nj, sj, width}.span();
    return {all.at, ni, si, 1, 0, all.width};
  }
};

// Whether rows of two sets of the same counts and strides share a byte, whose differences are those of (i, j) and (i', j').
inline bool dbs_like_rows_meet(const dbs_rows &a, const dbs_rows &b) {
  if (a.ni < a.nj) return dbs_like_rows_meet(a.turned(), b.turned());
  const __int128 step = a.si < 0 ? -a.si : a.si, most = a.ni - 1;
  const __int128 low = 1 - b.width, high = a.width - 1;  // b's row less a's, in bytes, where they meet
  const auto floor_div = [](__int128 x, __int128 y) { return x / y - (x % y < 0); };
  for (__int128 j = 1 - a.nj; j < a.nj; ++j) {
    const __int128 base = b.at - a.at + j * a.sj;
    if (step == 0 || most == 0) {
      if (low <= base && base <= high) return true;
      continue;
    }
    // some i from -most to most with low <= base + i step <= high
    __int128 first = -floor_div(base - low, step), last = floor_div(high - base, step);
    if (first < -most) first = -most;
    if (last > most) last = most;
    if (first <= last) return true;
  }
  return false;
}

// Whether rows of two sets of the same counts may share a byte: exact where their spans are apart or their strides are alike;
// where one stride is alike, the rows along the other are taken together, bytes between them included; else the spans decide.
inline bool dbs_rows_meet(dbs_rows a, dbs_rows b) {
  if (a.ni < 2) a.si = b.si = 0;
  if (a.nj < 2) a.sj = b.sj = 0;
  if (!dbs_like_rows_meet(a.span(), b.span())) return false;
  if (a.si == b.si && !dbs_like_rows_meet(a.joined(), b.joined())) return false;
  if (a.sj == b.sj && !dbs_like_rows_meet(a.turned().joined(), b.turned().joined())) return false;
  return a.si != b.si || a.sj != b.sj || dbs_like_rows_meet(a, b);  // the last, exact, takes longest: in steps over i or j
}

// whether rows of `width` elements at i * si + j * sj are disjoint because each i's rows end before the next i's begin
inline bool dbs_rows_apart(int64_t ni, int64_t si, int64_t nj, int64_t sj, int64_t width) {
  typedef __int128 wide;
  const wide i = si < 0 ? -(wide)si : si, j = sj < 0 ? -(wide)sj : sj;
  return (nj < 2 || j >= width) && (ni < 2 || i >= (nj - 1) * j + width);
}

// a barrier that waits for LDS only, not for loads from memory in flight
DBS_DEV void dbs_barrier_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
