// Argument marshalling of the decode-step entry points, in C++: the checks of a call's tensors cost 0.3 us here and 2 us (the
// logits' dozen 6 us) in Python, next to a launch of 2.8 us.  Nothing is computed: each function checks its tensors and
// calls the C ABI of include/dbs.h, whose functions bind() takes by address from the loaded libdbs.so.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

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
    return PyLong_FromLong(f());
  } catch (const failed &) {
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

// addresses of dbs_q4_product, dbs_q4_product_masked, dbs_q4_gated, dbs_logits_adjust, dbs_rope
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  try {
    if (n != 5) fail(PyExc_TypeError, "%zd arguments, expected 5", n);
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
                         METHOD(logits_adjust), METHOD(rope), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
