// pa_pycall.cpp -- argument marshalling of the windowed-attention and
// norm-rotation calls, as a CPython extension (_pycall.so).
//
// These calls are made per layer and step, and the smallest run for a few
// microseconds on the GPU: checked and passed on in Python, a call's arguments
// took 5 to 11 us, of which this leaves 2 to 4.  It knows torch by the public
// attributes of a tensor only (dtype, shape, get_device(), is_contiguous(),
// stride(), data_ptr()), so it is built without torch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <string.h>

#include "../../include/pa.h"

namespace {

// Set once by setup().
PyObject *g_tensor, *g_bf16, *g_f32, *g_i32, *g_i64, *g_u8;
PyObject *g_raw_stream, *g_current_device, *g_error;
// Interned attribute names.
PyObject *n_dtype, *n_shape, *n_get_device, *n_is_contiguous, *n_stride, *n_data_ptr, *n_stream;

constexpr int kMaxDims = 4;

struct Ref {  // an owned reference
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {}
  ~Ref() { Py_XDECREF(p); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

// The integers of a tuple; false with an error set.
bool read_ints(PyObject* tuple, long long* to, int n) {
  for (int i = 0; i < n; ++i) {
    to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (to[i] == -1 && PyErr_Occurred()) return false;
  }
  return true;
}

// Type, number of dimensions and CUDA device of an argument.
bool look(PyObject* t, const char* name, PyObject* dtype, int dims, long long* shape, int* device) {
  if (Py_TYPE(t) != reinterpret_cast<PyTypeObject*>(g_tensor)) {
    const int is = PyObject_IsInstance(t, g_tensor);
    if (is < 0) return false;
    if (!is) {
      PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
      return false;
    }
  }
  Ref dt(PyObject_GetAttr(t, n_dtype));
  if (!dt.p) return false;
  if (dt.p != dtype) {
    PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, dtype, dt.p);
    return false;
  }
  Ref dev(PyObject_CallMethodNoArgs(t, n_get_device));
  if (!dev.p) return false;
  *device = static_cast<int>(PyLong_AsLong(dev.p));
  if (*device < 0) {
    if (PyErr_Occurred()) return false;
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return false;
  }
  Ref sh(PyObject_GetAttr(t, n_shape));
  if (!sh.p) return false;
  if (!PyTuple_Check(sh.p) || PyTuple_GET_SIZE(sh.p) != dims) {
    PyErr_Format(PyExc_ValueError, "%s must have %d dims, got %S", name, dims, sh.p);
    return false;
  }
  return read_ints(sh.p, shape, dims);
}

bool address(PyObject* t, void** p) {
  Ref a(PyObject_CallMethodNoArgs(t, n_data_ptr));
  if (!a.p) return false;
  *p = PyLong_AsVoidPtr(a.p);
  return !PyErr_Occurred();
}

bool contiguous(PyObject* t, const char* name) {
  Ref c(PyObject_CallMethodNoArgs(t, n_is_contiguous));
  if (!c.p) return false;
  if (c.p != Py_True) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return false;
  }
  return true;
}

// The first tensor of a call: its shape and device are what others must have.
bool first(PyObject* t, const char* name, PyObject* dtype, int dims, long long* shape, int* device,
           void** p) {
  return look(t, name, dtype, dims, shape, device) && contiguous(t, name) && address(t, p);
}

bool same(const char* name, const long long* got, const long long* want, int dims, int device,
          int on) {
  if (memcmp(got, want, sizeof(long long) * dims) != 0) {
    char text[160];
    int at = 0;
    for (int i = 0; i < dims; ++i)
      at += PyOS_snprintf(text + at, sizeof text - at, "%s%lld", i ? ", " : "", want[i]);
    PyErr_Format(PyExc_ValueError, "%s must have shape (%s)", name, text);
    return false;
  }
  if (device != on) {
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, and other arguments on cuda:%d", name,
                 device, on);
    return false;
  }
  return true;
}

// A contiguous tensor of this type, shape and device.
bool tensor(PyObject* t, const char* name, PyObject* dtype, const long long* want, int dims,
            int on, void** p) {
  long long shape[kMaxDims];
  int device;
  return look(t, name, dtype, dims, shape, &device) &&
         same(name, shape, want, dims, device, on) && contiguous(t, name) && address(t, p);
}

// The same, or None (a null pointer).
bool optional(PyObject* t, const char* name, PyObject* dtype, const long long* want, int dims,
              int on, void** p) {
  *p = nullptr;
  return t == Py_None || tensor(t, name, dtype, want, dims, on, p);
}

// bf16 rows [tokens, heads, head_dim] at any token stride.  A single token's
// stride is never used: any view of one row will do.
bool rows(PyObject* t, const char* name, const long long* want, const long long* shape, int device,
          int on, void** p, long long* stride) {
  if (!same(name, shape, want, 3, device, on)) return false;
  Ref st(PyObject_CallMethodNoArgs(t, n_stride));
  long long s[3];
  if (!st.p || !read_ints(st.p, s, 3)) return false;
  if ((s[2] != 1 && shape[2] > 1) || (s[1] != shape[2] && shape[1] > 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous within a token", name);
    return false;
  }
  *stride = shape[0] > 1 ? s[0] : shape[1] * shape[2];
  return address(t, p);
}

bool whole(PyObject* v, const char* name, long long least, long long most, long long* out) {
  Ref n(PyNumber_Index(v));
  if (!n.p) return false;
  int over = 0;
  *out = PyLong_AsLongLongAndOverflow(n.p, &over);
  if (over || *out < least || *out > most) {
    PyErr_Clear();
    PyErr_Format(PyExc_ValueError, "%s must be in [%lld, %lld], got %S", name, least, most, v);
    return false;
  }
  return true;
}

bool real(PyObject* v, float* out) {
  const double d = PyFloat_AsDouble(v);
  if (d == -1.0 && PyErr_Occurred()) return false;
  *out = static_cast<float>(d);
  return true;
}

// A size that the C call takes as an int.
bool fits(long long n, const char* name) {
  if (n <= INT_MAX) return true;
  PyErr_Format(PyExc_ValueError, "%s has more than 2**31 - 1 entries", name);
  return false;
}

// The raw stream of a call whose tensors are on `device`: the current device.
bool queue(PyObject* stream, int device, void** out) {
  Ref cur(PyObject_CallNoArgs(g_current_device));
  if (!cur.p) return false;
  const long now = PyLong_AsLong(cur.p);
  if (now == -1 && PyErr_Occurred()) return false;
  if (now != device) {
    PyErr_Format(PyExc_ValueError, "tensors on cuda:%d, current device cuda:%ld", device, now);
    return false;
  }
  if (stream == Py_None) {
    Ref s(PyObject_CallOneArg(g_raw_stream, cur.p));
    if (!s.p) return false;
    *out = PyLong_AsVoidPtr(s.p);
  } else {
    Ref s(PyObject_GetAttr(stream, n_stream));
    if (!s.p) return false;
    *out = PyLong_AsVoidPtr(s.p);
  }
  return !PyErr_Occurred();
}

PyObject* done(const char* fn, int rc) {
  if (rc == PA_OK) Py_RETURN_NONE;
  Ref e(PyObject_CallFunction(g_error, "si", fn, rc));
  if (e.p) PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e.p)), e.p);
  return nullptr;
}

bool count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
  return false;
}

// decode_window(out, q, k_cache, v_cache, block_tables, seq_lens, window, sinks, scale, out_lse,
//               stream)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  long long qs[3], ks[4], bs[2], window, sinks;
  int dev, kdev, bdev;
  void *out, *q, *k, *v, *bt, *sl, *lse, *stream;
  float scale;
  if (!first(a[1], "q", g_bf16, 3, qs, &dev, &q) ||
      !look(a[2], "k_cache", g_bf16, 4, ks, &kdev) ||
      !look(a[4], "block_tables", g_i32, 2, bs, &bdev))
    return nullptr;
  const long long kv_want[4] = {ks[0], ks[1], ks[2], qs[2]}, bt_want[2] = {qs[0], bs[1]};
  if (!same("k_cache", ks, kv_want, 4, kdev, dev) || !contiguous(a[2], "k_cache") ||
      !address(a[2], &k) || !tensor(a[0], "out", g_bf16, qs, 3, dev, &out) ||
      !tensor(a[3], "v_cache", g_bf16, ks, 4, dev, &v) ||
      !same("block_tables", bs, bt_want, 2, bdev, dev) || !contiguous(a[4], "block_tables") ||
      !address(a[4], &bt) || !tensor(a[5], "seq_lens", g_i32, qs, 1, dev, &sl) ||
      !whole(a[6], "window", 1, INT_MAX, &window) || !whole(a[7], "sinks", 0, INT_MAX, &sinks) ||
      !real(a[8], &scale) || !optional(a[9], "out_lse", g_f32, qs, 2, dev, &lse) ||
      !fits(qs[0], "q") || !fits(qs[1], "q") || !fits(bs[1], "block_tables") ||
      !fits(ks[1], "k_cache") || !fits(ks[2], "k_cache") || !queue(a[10], dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pa_decode_window(out, q, k, v, static_cast<const int32_t*>(bt), static_cast<int>(bs[1]),
                        static_cast<const int32_t*>(sl), static_cast<int>(qs[0]),
                        static_cast<int>(qs[1]), static_cast<int>(ks[2]),
                        static_cast<int>(qs[2] > INT_MAX ? 0 : qs[2]), static_cast<int>(ks[1]),
                        ks[0], static_cast<int>(window), static_cast<int>(sinks), scale,
                        static_cast<float*>(lse), stream);
  Py_END_ALLOW_THREADS;
  return done("pa_decode_window", rc);
}

// prefill_window(out, q, k_cache, v_cache, block_tables, cu_q_lens, q_start_pos, seq_lens,
//                max_q_len, window, sinks, scale, out_lse, stream)
PyObject* prefill_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 14)) return nullptr;
  long long qs[3], ks[4], bs[2], cs[1], max_q, window, sinks;
  int dev, kdev, bdev, cdev;
  void *out, *q, *k, *v, *bt, *cu, *start, *sl, *lse, *stream;
  float scale;
  if (!first(a[1], "q", g_bf16, 3, qs, &dev, &q) ||
      !look(a[2], "k_cache", g_bf16, 4, ks, &kdev) ||
      !look(a[4], "block_tables", g_i32, 2, bs, &bdev) ||
      !look(a[5], "cu_q_lens", g_i32, 1, cs, &cdev))
    return nullptr;
  if (cs[0] < 1) {
    PyErr_SetString(PyExc_ValueError, "cu_q_lens must hold one more entry than there are chunks");
    return nullptr;
  }
  const long long chunks[1] = {cs[0] - 1};
  const long long kv_want[4] = {ks[0], ks[1], ks[2], qs[2]}, bt_want[2] = {chunks[0], bs[1]};
  if (!same("k_cache", ks, kv_want, 4, kdev, dev) || !contiguous(a[2], "k_cache") ||
      !address(a[2], &k) || !tensor(a[0], "out", g_bf16, qs, 3, dev, &out) ||
      !tensor(a[3], "v_cache", g_bf16, ks, 4, dev, &v) ||
      !same("block_tables", bs, bt_want, 2, bdev, dev) || !contiguous(a[4], "block_tables") ||
      !address(a[4], &bt) || !same("cu_q_lens", cs, cs, 1, cdev, dev) ||
      !contiguous(a[5], "cu_q_lens") || !address(a[5], &cu) ||
      !tensor(a[6], "q_start_pos", g_i32, chunks, 1, dev, &start) ||
      !tensor(a[7], "seq_lens", g_i32, chunks, 1, dev, &sl) ||
      !whole(a[8], "max_q_len", 0, INT_MAX, &max_q) ||
      !whole(a[9], "window", 1, INT_MAX, &window) || !whole(a[10], "sinks", 0, INT_MAX, &sinks) ||
      !real(a[11], &scale) || !optional(a[12], "out_lse", g_f32, qs, 2, dev, &lse) ||
      !fits(qs[0], "q") || !fits(qs[1], "q") || !fits(bs[1], "block_tables") ||
      !fits(ks[1], "k_cache") || !fits(ks[2], "k_cache") || !fits(chunks[0], "cu_q_lens") ||
      !queue(a[13], dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pa_prefill_window(
      out, q, k, v, static_cast<const int32_t*>(bt), static_cast<int>(bs[1]),
      static_cast<const int32_t*>(cu), static_cast<const int32_t*>(start),
      static_cast<const int32_t*>(sl), static_cast<int>(chunks[0]), static_cast<int>(qs[0]),
      static_cast<int>(max_q), static_cast<int>(qs[1]), static_cast<int>(ks[2]),
      static_cast<int>(qs[2] > INT_MAX ? 0 : qs[2]), static_cast<int>(ks[1]), ks[0],
      static_cast<int>(window), static_cast<int>(sinks), scale, static_cast<float*>(lse), stream);
  Py_END_ALLOW_THREADS;
  return done("pa_prefill_window", rc);
}

// norm_rope(q_out, k_out, q, k, v, positions, increments, k_cache, v_cache, slot_mapping,
//           k_scales, v_scales, q_weight, k_weight, eps, interleaved, rope_factor, stream, e4m3)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 19)) return nullptr;
  const int fp8 = PyObject_IsTrue(a[18]), il = PyObject_IsTrue(a[15]);
  if (fp8 < 0 || il < 0) return nullptr;
  long long qs[3], ks[3], vs[3], ps[4];
  int dev, kdev, vdev, pdev;
  void *q_out, *k_out, *q, *k, *v = nullptr, *pos = nullptr, *inc = nullptr, *kc = nullptr,
                                *vc = nullptr, *slots = nullptr, *sk = nullptr, *sv = nullptr,
                                *qw, *kw, *stream;
  long long q_stride, k_stride, v_stride = 0, nb = 0, bs = 0, rot = 0;
  float eps, factor;
  if (!look(a[2], "q", g_bf16, 3, qs, &dev) || !look(a[3], "k", g_bf16, 3, ks, &kdev))
    return nullptr;
  const long long kv_want[3] = {qs[0], ks[1], qs[2]};
  if (!rows(a[2], "q", qs, qs, dev, dev, &q, &q_stride) ||
      !rows(a[3], "k", kv_want, ks, kdev, dev, &k, &k_stride))
    return nullptr;
  if (fp8 || a[7] != Py_None || a[8] != Py_None) {
    PyObject* type = fp8 ? g_u8 : g_bf16;
    if (!look(a[4], "v", g_bf16, 3, vs, &vdev) ||
        !rows(a[4], "v", kv_want, vs, vdev, dev, &v, &v_stride) ||
        !look(a[7], "k_cache", type, 4, ps, &pdev))
      return nullptr;
    nb = ps[0];
    bs = ps[1];
    const long long pool[4] = {nb, bs, ks[1], qs[2]};
    if (!same("k_cache", ps, pool, 4, pdev, dev) || !contiguous(a[7], "k_cache") ||
        !address(a[7], &kc) || !tensor(a[8], "v_cache", type, pool, 4, dev, &vc) ||
        !tensor(a[9], "slot_mapping", g_i64, qs, 1, dev, &slots))
      return nullptr;
  }
  if (fp8 && (!tensor(a[10], "k_scales", g_f32, ks + 1, 1, dev, &sk) ||
              !tensor(a[11], "v_scales", g_f32, ks + 1, 1, dev, &sv)))
    return nullptr;
  if (a[6] != Py_None) {
    long long is[1];
    int idev;
    if (!look(a[6], "increments", g_i64, 1, is, &idev) ||
        !same("increments", is, is, 1, idev, dev) || !contiguous(a[6], "increments") ||
        !address(a[6], &inc) || !tensor(a[5], "positions", g_i64, qs, 1, dev, &pos))
      return nullptr;
    rot = 2 * (is[0] < INT_MAX / 2 ? is[0] : INT_MAX / 2);  // (a huge one is refused below)
  }
  if (!tensor(a[0], "q_out", g_bf16, qs, 3, dev, &q_out) ||
      !optional(a[1], "k_out", g_bf16, kv_want, 3, dev, &k_out) ||
      !optional(a[12], "q_weight", g_f32, qs + 2, 1, dev, &qw) ||
      !optional(a[13], "k_weight", g_f32, qs + 2, 1, dev, &kw) || !real(a[14], &eps) ||
      !real(a[16], &factor) || !fits(qs[0], "q") || !fits(qs[1], "q") || !fits(qs[2], "q") ||
      !fits(ks[1], "k") || !fits(bs, "k_cache") || !queue(a[17], dev, &stream))
    return nullptr;
  const int T = static_cast<int>(qs[0]), Hq = static_cast<int>(qs[1]),
            Hkv = static_cast<int>(ks[1]), D = static_cast<int>(qs[2]);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  if (fp8)
    rc = pa_qk_norm_rope_cache_fp8(
        q_out, k_out, q, k, v, q_stride, k_stride, v_stride, static_cast<float*>(qw),
        static_cast<float*>(kw), eps, static_cast<int64_t*>(pos), static_cast<int64_t*>(inc),
        static_cast<int>(rot), il, factor, kc, vc, static_cast<int64_t*>(slots),
        static_cast<float*>(sk), static_cast<float*>(sv), T, Hq, Hkv, D, static_cast<int>(bs), nb,
        stream);
  else
    rc = pa_qk_norm_rope_cache(
        q_out, k_out, q, k, v, q_stride, k_stride, v_stride, static_cast<float*>(qw),
        static_cast<float*>(kw), eps, static_cast<int64_t*>(pos), static_cast<int64_t*>(inc),
        static_cast<int>(rot), il, factor, kc, vc, static_cast<int64_t*>(slots), T, Hq, Hkv, D,
        static_cast<int>(bs), nb, stream);
  Py_END_ALLOW_THREADS;
  return done(fp8 ? "pa_qk_norm_rope_cache_fp8" : "pa_qk_norm_rope_cache", rc);
}

// setup(torch.Tensor, bfloat16, float32, int32, int64, uint8, raw stream of a device, current
//       device, the exception class of a refused call)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  PyObject** to[9] = {&g_tensor, &g_bf16, &g_f32, &g_i32, &g_i64, &g_u8, &g_raw_stream,
                      &g_current_device, &g_error};
  for (int i = 0; i < 9; ++i) {
    Py_INCREF(a[i]);
    Py_XDECREF(*to[i]);
    *to[i] = a[i];
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(setup)), METH_FASTCALL, nullptr},
    {"decode_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_window)),
     METH_FASTCALL, nullptr},
    {"prefill_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefill_window)),
     METH_FASTCALL, nullptr},
    {"norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rope)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycall(void) {
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&n_dtype, "dtype"},   {&n_shape, "shape"},       {&n_get_device, "get_device"},
               {&n_is_contiguous, "is_contiguous"}, {&n_stride, "stride"},
               {&n_data_ptr, "data_ptr"}, {&n_stream, "cuda_stream"}};
  for (auto& x : names)
    if (!(*x.to = PyUnicode_InternFromString(x.name))) return nullptr;
  return PyModule_Create(&module);
}
