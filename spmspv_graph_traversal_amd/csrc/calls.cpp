// Argument marshalling of the decode-step entry points, in C++: the checks of a call's tensors cost 0.3 us here and 2 us (the
// logits' dozen 6 us) in Python, next to a launch of 2.8 us.  Nothing is computed: each function checks its tensors and
// calls the C ABI of include/dbs.h, whose functions bind() takes by address from the loaded libdbs.so.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>

#include <c10/hip/HIPCachingAllocator.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dbs.h"

namespace {

decltype(&dbs_q4_product) f_product;
decltype(&dbs_q4_product_masked) f_masked;
decltype(&dbs_q4_gated) f_gated;
decltype(&dbs_logits_adjust) f_logits;
decltype(&dbs_rope) f_rope;
decltype(&dbs_norm_rope) f_norm;
decltype(&dbs_kv4_page_bytes) f_page_bytes;
decltype(&dbs_kv4_store) f_store;
decltype(&dbs_kv4_attention_workspace) f_workspace;
decltype(&dbs_kv4_attention) f_attention;

// A Python exception is set where a check fails.
struct failed {};
template <class... A>
[[noreturn]] void fail(PyObject *type, const char *format, A... a) {
  PyErr_Format(type, format, a...);
  throw failed();
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw failed();
  return v;
}
// a value of an enum
template <class E>
E choice(PyObject *o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, "%lld is no choice", (long long)v);
  return (E)v;
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw failed();
  return v;
}
// handle.value of a freed matrix is None
void *pointer(PyObject *o) {
  if (o == Py_None) return nullptr;
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw failed();
  return p;
}

struct call {
  int device;
  void *stream;
  // `tensor` tells the device: it has to be the current one
  call(PyObject *tensor, const char *name, PyObject *given) {
    if (!THPVariable_Check(tensor) || !THPVariable_Unpack(tensor).is_cuda())
      fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
    device = c10::hip::current_device();
    if (THPVariable_Unpack(tensor).get_device() != device)
      fail(PyExc_ValueError, "%s is on device %d, the call runs on the current device, %d", name,
           (int)THPVariable_Unpack(tensor).get_device(), device);
    if (given == Py_None) {
      stream = c10::hip::getCurrentHIPStream(device).stream();
    } else {
      PyObject *raw = PyObject_GetAttrString(given, "cuda_stream");
      if (!raw) throw failed();
      stream = PyLong_AsVoidPtr(raw);
      Py_DECREF(raw);
      if (!stream && PyErr_Occurred()) throw failed();
      PyObject *at = PyObject_GetAttrString(given, "device_index");
      if (at) {
        const long index = PyLong_AsLong(at);
        Py_DECREF(at);
        if (index == -1 && PyErr_Occurred()) throw failed();
        if (index != device)
          fail(PyExc_ValueError, "the stream is on device %ld, the call runs on the current device, %d", index, device);
      } else {
        PyErr_Clear();
      }
    }
  }
  const at::Tensor &tensor(PyObject *o, const char *name) const {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.get_device() != device)
      fail(PyExc_ValueError, "%s is on device %d, the call runs on the current device, %d", name, (int)t.get_device(), device);
    return t;
  }
};

dbs_dtype vector_type(const at::Tensor &t, const char *name) {
  if (t.scalar_type() == at::kFloat) return DBS_F32;
  if (t.scalar_type() == at::kBFloat16) return DBS_BF16;
  fail(PyExc_TypeError, "%s has dtype %s, expected float32 or bfloat16", name, c10::toString(t.scalar_type()));
}

// a vector [width] or rows [rows, width] with contiguous elements and any row stride
struct rows {
  int64_t count, ld;
  dbs_dtype type;
  void *p;
  rows(const call &c, PyObject *o, const char *name, int64_t width, const char *what) {
    const at::Tensor &t = c.tensor(o, name);
    type = vector_type(t, name);
    const int64_t nd = t.dim();
    if (nd < 1 || nd > 2 || (width >= 0 && t.size(nd - 1) != width))
      fail(PyExc_ValueError, "%s must be [%lld] or [%s, %lld]", name, (long long)width, what, (long long)width);
    const int64_t w = t.size(nd - 1);
    count = nd == 2 ? t.size(0) : 1;
    ld = count > 1 ? t.stride(0) : w;
    if (t.stride(nd - 1) != 1 && w > 1) fail(PyExc_ValueError, "%s must have contiguous rows", name);
    if (ld < w) fail(PyExc_ValueError, "%s: rows overlap (row stride %lld < %lld)", name, (long long)ld, (long long)w);
    if (count > INT32_MAX || w > INT32_MAX) fail(PyExc_ValueError, "%s is too large", name);
    p = t.data_ptr();
  }
};

// words of a bit mask of [rows, width]; [words] for one row
struct mask_rows {
  int64_t ld;
  const uint32_t *p;
  mask_rows(const call &c, PyObject *o, int64_t count, int64_t width) {
    const at::Tensor &t = c.tensor(o, "the mask");
    if (t.scalar_type() != at::kInt && t.scalar_type() != at::kUInt32)
      fail(PyExc_TypeError, "the mask has dtype %s, expected int32 or uint32 words", c10::toString(t.scalar_type()));
    const int64_t words = (width + 31) / 32, nd = t.dim();
    const bool fits = nd == 2 ? t.size(0) == count && t.size(1) == words : nd == 1 && count == 1 && t.size(0) == words;
    if (!fits) fail(PyExc_ValueError, "the mask must be [%lld, %lld]", (long long)count, (long long)words);
    if (t.stride(nd - 1) != 1 && words > 1) fail(PyExc_ValueError, "the mask must have contiguous rows");
    ld = count > 1 ? t.stride(0) : words;
    if (ld < words) fail(PyExc_ValueError, "mask rows overlap");
    p = (const uint32_t *)t.data_ptr();
  }
};

// a contiguous list of `count` elements (-1: any number), or None
template <class T>
const T *list(const call &c, PyObject *o, const char *name, at::ScalarType type, int64_t count, int64_t *length = nullptr) {
  if (o == Py_None) return nullptr;
  const at::Tensor &t = c.tensor(o, name);
  if (t.scalar_type() != type || !t.is_contiguous())
    fail(PyExc_TypeError, "%s must be contiguous %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  if (count >= 0 && t.numel() != count)
    fail(PyExc_ValueError, "%s has %lld elements, expected %lld", name, (long long)t.numel(), (long long)count);
  if (length) *length = t.numel();
  return (const T *)t.data_ptr();
}

template <class F>
PyObject *status(F f) {
  try {
    return PyLong_FromLongLong(f());
  } catch (const failed &) {
  } catch (const c10::OutOfMemoryError &e) {
    PyObject *const torch = PyImport_ImportModule("torch"), *const type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// the library's call without the interpreter's lock: a launch waits while its queue is full
template <class F, class... A>
dbs_status unlocked(F f, A... a) {
  PyThreadState *const thread = PyEval_SaveThread();
  const dbs_status st = f(a...);
  PyEval_RestoreThread(thread);
  return st;
}

void need(Py_ssize_t have, Py_ssize_t want) {
  if (have != want) fail(PyExc_TypeError, "%zd arguments, expected %zd", have, want);
  if (!f_product) fail(PyExc_RuntimeError, "not bound to the library");
}

void same_tokens(const rows &x, const rows &y) {
  if (x.count != y.count) fail(PyExc_ValueError, "x has %lld tokens, y %lld", (long long)x.count, (long long)y.count);
}

// handle, m, n, x, y, stream
PyObject *q4_product(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&] {
    need(n, 6);
    const call c(a[4], "y", a[5]);
    const rows x(c, a[3], "x", integer(a[2]), "tokens"), y(c, a[4], "y", integer(a[1]), "tokens");
    same_tokens(x, y);
    return unlocked(f_product, (dbs_q4_handle)pointer(a[0]), (int32_t)x.count, x.p, x.type, x.ld, y.p, y.type, y.ld,
                    c.stream);
  });
}

// handle, m, n, x, mask, fill, y, stream
PyObject *q4_product_masked(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&] {
    need(n, 8);
    const call c(a[6], "y", a[7]);
    const rows x(c, a[3], "x", integer(a[2]), "tokens"), y(c, a[6], "y", integer(a[1]), "tokens");
    same_tokens(x, y);
    const mask_rows m(c, a[4], x.count, integer(a[1]));
    return unlocked(f_masked, (dbs_q4_handle)pointer(a[0]), (int32_t)x.count, x.p, x.type, x.ld, m.p, m.ld,
                    (float)number(a[5]), y.p, y.type, y.ld, c.stream);
  });
}

// gate, up, m, n, x, activation, y, stream
PyObject *q4_gated(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&] {
    need(n, 8);
    const call c(a[6], "y", a[7]);
    const rows x(c, a[4], "x", integer(a[3]), "tokens"), y(c, a[6], "y", integer(a[2]), "tokens");
    same_tokens(x, y);
    return unlocked(f_gated, (dbs_q4_handle)pointer(a[0]), (dbs_q4_handle)pointer(a[1]), choice<dbs_activation>(a[5]),
                    (int32_t)x.count, x.p, x.type, x.ld, y.p, y.type, y.ld, c.stream);
  });
}

// logits, out, hist_ptr, hist, hist_new, repetition, frequency, presence, bias_ptr, bias_idx, bias_val, mask, stream
PyObject *logits_adjust(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&] {
    need(n, 13);
    const call c(a[1], "out", a[12]);
    const rows l(c, a[0], "logits", -1, "rows");
    const at::Tensor &t = THPVariable_Unpack(a[0]);
    const int64_t vocab = t.size(t.dim() - 1);
    const rows o(c, a[1], "out", vocab, "rows");
    if (l.count != o.count)
      fail(PyExc_ValueError, "logits have %lld rows, out %lld", (long long)l.count, (long long)o.count);
    if ((a[2] == Py_None) != (a[3] == Py_None)) fail(PyExc_ValueError, "hist_ptr and hist go together");
    if ((a[8] == Py_None) != (a[9] == Py_None) || (a[9] == Py_None) != (a[10] == Py_None))
      fail(PyExc_ValueError, "bias_ptr, bias_idx and bias_val go together");
    dbs_logits_params p = {};
    p.hist_ptr = list<int32_t>(c, a[2], "hist_ptr", at::kInt, l.count + 1);
    p.hist = list<int32_t>(c, a[3], "hist", at::kInt, -1, &p.hist_len);
    p.hist_new = list<int32_t>(c, a[4], "hist_new", at::kInt, l.count);
    p.repetition = list<float>(c, a[5], "repetition", at::kFloat, l.count);
    p.frequency = list<float>(c, a[6], "frequency", at::kFloat, l.count);
    p.presence = list<float>(c, a[7], "presence", at::kFloat, l.count);
    p.bias_ptr = list<int32_t>(c, a[8], "bias_ptr", at::kInt, l.count + 1);
    p.bias_idx = list<int32_t>(c, a[9], "bias_idx", at::kInt, -1, &p.bias_len);
    p.bias_val = list<float>(c, a[10], "bias_val", at::kFloat, p.bias_len);
    if (a[11] != Py_None) {
      const mask_rows m(c, a[11], l.count, vocab);
      p.mask = m.p;
      p.ldmask = m.ld;
    }
    return unlocked(f_logits, (int32_t)l.count, (int32_t)vocab, l.p, l.type, l.ld, &p, o.p, o.type, o.ld, c.stream);
  });
}

// x, pos, freq, out, layout, scale, inverse, stream
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&] {
    need(n, 8);
    const call c(a[3], "out", a[7]);
    const at::Tensor &x = c.tensor(a[0], "x"), &o = c.tensor(a[3], "out");
    if (x.dim() != 3 || o.dim() != 3 || x.sizes() != o.sizes())
      fail(PyExc_ValueError, "x and out must be [tokens, heads, head_dim] of one shape");
    const dbs_dtype xt = vector_type(x, "x"), ot = vector_type(o, "out");
    if (x.size(2) > 1 && (x.stride(2) != 1 || o.stride(2) != 1))
      fail(PyExc_ValueError, "x and out must have contiguous heads");
    if (x.size(0) > INT32_MAX || x.size(1) > INT32_MAX || x.size(2) > INT32_MAX) fail(PyExc_ValueError, "x is too large");
    if (a[1] == Py_None || a[2] == Py_None) fail(PyExc_TypeError, "pos and freq must be CUDA tensors");
    int64_t pairs = 0;
    const int32_t *pos = list<int32_t>(c, a[1], "pos", at::kInt, x.size(0));
    const double *freq = list<double>(c, a[2], "freq", at::kDouble, -1, &pairs);
    if (pairs > INT32_MAX / 2) fail(PyExc_ValueError, "freq is too large");
    const int inverse = PyObject_IsTrue(a[6]);
    if (inverse < 0) throw failed();
    return unlocked(f_rope, (int32_t)x.size(0), (int32_t)x.size(1), (int32_t)x.size(2), (int32_t)(2 * pairs),
                    choice<dbs_rope_layout>(a[4]), pos, freq, (float)number(a[5]), inverse, x.data_ptr(), xt, x.stride(0),
                    x.stride(1), o.data_ptr(), ot, o.stride(0), o.stride(1), c.stream);
  });
}

// heads [tokens, heads, head_dim] with contiguous elements and any other strides; None where that is allowed
struct heads {
  int64_t tokens = 0, count = 0, dim = 0, st = 0, sh = 0;
  dbs_dtype type = DBS_F32;
  void *p = nullptr;
  heads(const call &c, PyObject *o, const char *name, bool optional = false) {
    if (optional && o == Py_None) return;
    const at::Tensor &t = c.tensor(o, name);
    type = vector_type(t, name);
    if (t.dim() != 3) fail(PyExc_ValueError, "%s must be [tokens, heads, head_dim]", name);
    if (t.size(2) > 1 && t.numel() > 0 && t.stride(2) != 1) fail(PyExc_ValueError, "%s must have contiguous heads", name);
    tokens = t.size(0);
    count = t.size(1);
    dim = t.size(2);
    if (tokens > INT32_MAX || count > INT32_MAX || dim > INT32_MAX) fail(PyExc_ValueError, "%s is too large", name);
    st = t.stride(0);
    sh = t.stride(1);
    p = t.data_ptr();
  }
  void like(const heads &x, const char *name, const char *other) const {
    if (tokens != x.tokens || count != x.count || dim != x.dim) fail(PyExc_ValueError, "%s and %s must be of one shape", name, other);
  }
};

int32_t small(PyObject *o, const char *name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, "%s is out of range", name);
  return (int32_t)v;
}

// q, k, q_weight, k_weight, pos, freq, q_out, k_out, eps, layout, scale, stream
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&] {
    need(n, 12);
    const call c(a[6], "q_out", a[11]);
    const heads q(c, a[0], "q"), k(c, a[1], "k", true), qo(c, a[6], "q_out"), ko(c, a[7], "k_out", true);
    const bool two = a[1] != Py_None;
    if (two != (a[7] != Py_None)) fail(PyExc_ValueError, "k and k_out go together");
    if (!two && a[3] != Py_None) fail(PyExc_ValueError, "k_weight without k");
    qo.like(q, "q", "q_out");
    if (two) {
      ko.like(k, "k", "k_out");
      if (k.tokens != q.tokens || k.dim != q.dim) fail(PyExc_ValueError, "q and k have the same tokens and head_dim");
      if (k.type != q.type || ko.type != qo.type) fail(PyExc_TypeError, "q and k, and their outputs, have the same dtype");
    }
    if (a[4] == Py_None || a[5] == Py_None) fail(PyExc_TypeError, "pos and freq must be CUDA tensors");
    int64_t pairs = 0;
    const int32_t *pos = list<int32_t>(c, a[4], "pos", at::kInt, q.tokens);
    const double *freq = list<double>(c, a[5], "freq", at::kDouble, -1, &pairs);
    if (pairs > INT32_MAX / 2) fail(PyExc_ValueError, "freq is too large");
    dbs_dtype weight_type = DBS_F32;
    const void *weight[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
      if (a[2 + i] == Py_None) continue;
      const char *const name = i ? "k_weight" : "q_weight";
      const at::Tensor &t = c.tensor(a[2 + i], name);
      const dbs_dtype type = vector_type(t, name);
      if (!t.is_contiguous() || t.dim() != 1 || t.size(0) != q.dim) fail(PyExc_ValueError, "%s must be [%lld], contiguous", name, (long long)q.dim);
      if (i && weight[0] && type != weight_type) fail(PyExc_TypeError, "the weights have the same dtype");
      weight_type = type;
      weight[i] = t.data_ptr();
    }
    const dbs_norm_part parts[2] = {{q.p, q.st, q.sh, qo.p, qo.st, qo.sh, (int32_t)q.count, weight[0]},
                                    {k.p, k.st, k.sh, ko.p, ko.st, ko.sh, (int32_t)k.count, weight[1]}};
    return unlocked(f_norm, (int32_t)q.tokens, (int32_t)q.dim, (int32_t)(2 * pairs), choice<dbs_rope_layout>(a[9]), pos, freq,
                    (float)number(a[10]), (float)number(a[8]), &parts[0], two ? 2 : 1, q.type, qo.type, weight_type, c.stream);
  });
}

// pool, key_heads, head_dim, group, page_tokens, table, lens, and new_ptr
struct cache {
  dbs_kv4_cache v = {};
  cache(const call &c, PyObject *const *a, PyObject *new_ptr) {
    const at::Tensor &pool = c.tensor(a[0], "the pool"), &table = c.tensor(a[5], "table");
    if (pool.scalar_type() != at::kByte || pool.dim() != 2 || (pool.size(1) > 1 && pool.stride(1) != 1))
      fail(PyExc_TypeError, "the pool must be uint8 [pages, bytes] with contiguous pages");
    v.key_heads = small(a[1], "key_heads");
    v.head_dim = small(a[2], "head_dim");
    v.group = small(a[3], "group");
    v.page_tokens = small(a[4], "page_tokens");
    if (pool.size(0) > INT32_MAX) fail(PyExc_ValueError, "the pool has too many pages");
    v.pool = pool.data_ptr();
    v.pages = (int32_t)pool.size(0);
    int64_t bytes = 0;
    if (f_page_bytes(v.key_heads, v.head_dim, v.group, v.page_tokens, &bytes) != DBS_OK)
      fail(PyExc_ValueError, "no cache of %d heads of %d in groups of %d and pages of %d tokens", (int)v.key_heads, (int)v.head_dim,
           (int)v.group, (int)v.page_tokens);
    if (pool.size(1) < bytes) fail(PyExc_ValueError, "pages have %lld bytes, %lld are needed", (long long)pool.size(1), (long long)bytes);
    v.page_stride = v.pages > 1 ? pool.stride(0) : bytes;
    if (v.page_stride < bytes) fail(PyExc_ValueError, "pages of the pool overlap");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
      fail(PyExc_TypeError, "table must be int32 [sequences, pages] with contiguous rows");
    if (table.size(0) > INT32_MAX || table.size(1) > INT32_MAX) fail(PyExc_ValueError, "table is too large");
    v.sequences = (int32_t)table.size(0);
    v.table_pages = (int32_t)table.size(1);
    v.ldtable = v.sequences > 1 ? table.stride(0) : v.table_pages;
    v.table = (const int32_t *)table.data_ptr();
    if (a[6] == Py_None) fail(PyExc_TypeError, "lens must be a CUDA tensor");
    v.lens = list<int32_t>(c, a[6], "lens", at::kInt, v.sequences);
    v.new_ptr = list<int32_t>(c, new_ptr, "new_ptr", at::kInt, (int64_t)v.sequences + 1);
  }
  void takes(const heads &x, const char *name) const {
    if (x.dim != v.head_dim) fail(PyExc_ValueError, "%s has heads of %lld, the cache of %d", name, (long long)x.dim, (int)v.head_dim);
    if (!v.new_ptr && v.sequences > 0 && x.tokens % v.sequences)
      fail(PyExc_ValueError, "%lld tokens of %d sequences: new_ptr is needed", (long long)x.tokens, (int)v.sequences);
  }
};

// pool, key_heads, head_dim, group, page_tokens, table, lens, k, v, new_ptr, k_out, v_out, stream
PyObject *kv4_store(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&] {
    need(n, 13);
    const call c(a[0], "the pool", a[12]);
    const cache s(c, a, a[9]);
    const heads k(c, a[7], "k"), v(c, a[8], "v"), ko(c, a[10], "k_out", true), vo(c, a[11], "v_out", true);
    s.takes(k, "k");
    v.like(k, "k", "v");
    if (k.count != s.v.key_heads) fail(PyExc_ValueError, "k has %lld heads, the cache %d", (long long)k.count, (int)s.v.key_heads);
    if (v.type != k.type) fail(PyExc_TypeError, "k and v have the same dtype");
    if (ko.p || a[10] != Py_None) ko.like(k, "k", "k_out");
    if (vo.p || a[11] != Py_None) vo.like(v, "v", "v_out");
    if (a[10] != Py_None && a[11] != Py_None && ko.type != vo.type) fail(PyExc_TypeError, "k_out and v_out have the same dtype");
    return unlocked(f_store, &s.v, (int32_t)k.tokens, k.p, k.st, k.sh, v.p, v.st, v.sh, k.type, ko.p, ko.st, ko.sh, vo.p, vo.st, vo.sh,
                    a[10] != Py_None ? ko.type : vo.type, c.stream);
  });
}

// pool, key_heads, head_dim, group, page_tokens, table, lens, q, out, new_ptr, window, sinks, scale, max_len, workspace, stream
PyObject *kv4_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&]() -> long {
    need(n, 16);
    const call c(a[8], "out", a[15]);
    const cache s(c, a, a[9]);
    const heads q(c, a[7], "q"), o(c, a[8], "out");
    s.takes(q, "q");
    o.like(q, "q", "out");
    const int32_t window = small(a[10], "window"), sinks = small(a[11], "sinks"), max_len = small(a[13], "max_len");
    const float scale = a[12] == Py_None ? (float)(1.0 / std::sqrt((double)q.dim)) : (float)number(a[12]);
    int64_t bytes = 0;
    void *space = nullptr;
    void *own = nullptr;
    if (a[14] == Py_None) {
      const dbs_status st = f_workspace(&s.v, (int32_t)q.tokens, (int32_t)q.count, q.type, o.type, window, sinks, max_len, &bytes);
      if (st != DBS_OK) return st;
      // from the given stream's memory, and given back to it: what it runs later may have it
      if (bytes > 0) own = c10::hip::HIPCachingAllocator::raw_alloc_with_stream((size_t)bytes, (hipStream_t)c.stream);
      space = own;
    } else {
      const at::Tensor &t = c.tensor(a[14], "workspace");
      if (t.scalar_type() != at::kByte || !t.is_contiguous()) fail(PyExc_TypeError, "workspace must be contiguous uint8");
      bytes = t.numel();
      space = t.data_ptr();
    }
    const dbs_status st = unlocked(f_attention, &s.v, (int32_t)q.tokens, (int32_t)q.count, q.p, q.type, q.st, q.sh, o.p, o.type, o.st, o.sh,
                                   scale, window, sinks, max_len, space, bytes, c.stream);
    if (own) c10::hip::HIPCachingAllocator::raw_delete(own);
    return st;
  });
}

// pool, key_heads, head_dim, group, page_tokens, table, lens, q, out, new_ptr, window, sinks, max_len
PyObject *kv4_workspace(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status([&] {
    need(n, 13);
    const call c(a[8], "out", Py_None);
    const cache s(c, a, a[9]);
    const heads q(c, a[7], "q"), o(c, a[8], "out");
    s.takes(q, "q");
    o.like(q, "q", "out");
    int64_t bytes = 0;
    const dbs_status st = f_workspace(&s.v, (int32_t)q.tokens, (int32_t)q.count, q.type, o.type, small(a[10], "window"), small(a[11], "sinks"),
                                      small(a[12], "max_len"), &bytes);
    if (st != DBS_OK) fail(PyExc_ValueError, "no call of these arguments (status %d)", (int)st);
    return bytes;
  });
}

// addresses of dbs_q4_product, dbs_q4_product_masked, dbs_q4_gated, dbs_logits_adjust, dbs_rope, dbs_norm_rope,
// dbs_kv4_page_bytes, dbs_kv4_store, dbs_kv4_attention_workspace, dbs_kv4_attention
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  try {
    if (n != 10) fail(PyExc_TypeError, "%zd arguments, expected 10", n);
    f_norm = (decltype(f_norm))pointer(a[5]);
    f_page_bytes = (decltype(f_page_bytes))pointer(a[6]);
    f_store = (decltype(f_store))pointer(a[7]);
    f_workspace = (decltype(f_workspace))pointer(a[8]);
    f_attention = (decltype(f_attention))pointer(a[9]);
    f_masked = (decltype(f_masked))pointer(a[1]);
    f_gated = (decltype(f_gated))pointer(a[2]);
    f_logits = (decltype(f_logits))pointer(a[3]);
    f_rope = (decltype(f_rope))pointer(a[4]);
    f_product = (decltype(f_product))pointer(a[0]);
  } catch (const failed &) {
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(q4_product), METHOD(q4_product_masked), METHOD(q4_gated),
                         METHOD(logits_adjust), METHOD(rope), METHOD(norm_rope),
                         METHOD(kv4_store), METHOD(kv4_attention), METHOD(kv4_workspace), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
