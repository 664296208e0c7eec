// pa_pycall.cpp -- argument marshalling of the windowed-attention and
// norm-rotation calls, as a CPython extension (_pycall.so).
//
// These calls are made per layer and step, and the smallest run for a few
// microseconds on the GPU: checked and passed on in Python, a call's arguments
// took 5 to 11 us; read through the tensors' Python attributes, 2 to 4; read
// from the tensors themselves, as here, below one.
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits.h>

#include <exception>

#include "../../include/pa.h"

namespace {

PyObject* g_error;   // the exception class of a refused call, set once by setup()
PyObject* n_stream;  // interned: "cuda_stream"

using Shape = at::IntArrayRef;

struct Ref {  // an owned reference
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {}
  ~Ref() { Py_XDECREF(p); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

// A CUDA tensor of this type and number of dimensions; null with an error set.
const at::Tensor* look(PyObject* o, const char* name, at::ScalarType type, int dims) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor of %s, got %s", name, at::toString(type),
                 at::toString(t.scalar_type()));
    return nullptr;
  }
  if (!t.is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return nullptr;
  }
  if (t.dim() != dims) {
    PyErr_Format(PyExc_ValueError, "%s must have %d dims, got %lld", name, dims,
                 static_cast<long long>(t.dim()));
    return nullptr;
  }
  return &t;
}

bool contiguous(const at::Tensor& t, const char* name) {
  if (t.is_contiguous()) return true;
  PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
  return false;
}

// Shape and device as another argument has them.
bool same(const at::Tensor& t, const char* name, Shape want, int device) {
  if (t.sizes() != want) {
    char text[160];
    int at = 0;
    text[0] = 0;
    for (size_t i = 0; i < want.size(); ++i)
      at += PyOS_snprintf(text + at, sizeof text - at, "%s%lld", i ? ", " : "",
                          static_cast<long long>(want[i]));
    PyErr_Format(PyExc_ValueError, "%s must have shape (%s)", name, text);
    return false;
  }
  if (t.get_device() != device) {
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, and other arguments on cuda:%d", name,
                 static_cast<int>(t.get_device()), device);
    return false;
  }
  return true;
}

// A contiguous tensor of this type, shape and device.
bool tensor(PyObject* o, const char* name, at::ScalarType type, Shape want, int device, void** p) {
  const at::Tensor* t = look(o, name, type, static_cast<int>(want.size()));
  if (!t || !same(*t, name, want, device) || !contiguous(*t, name)) return false;
  *p = t->data_ptr();
  return true;
}

// The same, or None (a null pointer).
bool optional(PyObject* o, const char* name, at::ScalarType type, Shape want, int device,
              void** p) {
  *p = nullptr;
  return o == Py_None || tensor(o, name, type, want, device, p);
}

// bf16 rows [tokens, heads, head_dim] at any token stride.  A single token's
// stride is never used: any view of one row will do.
bool rows(const at::Tensor& t, const char* name, Shape want, int device, void** p,
          int64_t* stride) {
  if (!same(t, name, want, device)) return false;
  const Shape n = t.sizes(), s = t.strides();
  if ((s[2] != 1 && n[2] > 1) || (s[1] != n[2] && n[1] > 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous within a token", name);
    return false;
  }
  *stride = n[0] > 1 ? s[0] : n[1] * n[2];
  *p = t.data_ptr();
  return true;
}

bool whole(PyObject* v, const char* name, long long least, long long most, int* out) {
  Ref n(PyNumber_Index(v));
  if (!n.p) return false;
  int over = 0;
  const long long x = PyLong_AsLongLongAndOverflow(n.p, &over);
  if (over || x < least || x > most) {
    PyErr_Clear();
    PyErr_Format(PyExc_ValueError, "%s must be in [%lld, %lld], got %S", name, least, most, v);
    return false;
  }
  *out = static_cast<int>(x);
  return true;
}

bool real(PyObject* v, float* out) {
  const double d = PyFloat_AsDouble(v);
  if (d == -1.0 && PyErr_Occurred()) return false;
  *out = static_cast<float>(d);
  return true;
}

// A size that the C call takes as an int.
bool fits(int64_t n, const char* name) {
  if (n <= INT_MAX) return true;
  PyErr_Format(PyExc_ValueError, "%s has more than 2**31 - 1 entries", name);
  return false;
}

// The raw stream of a call whose tensors are on `device`: the current device.
bool queue(PyObject* stream, int device, void** out) {
  const int now = c10::cuda::current_device();
  if (now != device) {
    PyErr_Format(PyExc_ValueError, "tensors on cuda:%d, current device cuda:%d", device, now);
    return false;
  }
  if (stream == Py_None) {
    *out = c10::cuda::getCurrentCUDAStream(now).stream();
    return true;
  }
  Ref s(PyObject_GetAttr(stream, n_stream));
  if (!s.p) return false;
  *out = PyLong_AsVoidPtr(s.p);
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

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt,
                         kI64 = at::kLong, kU8 = at::kByte;

// decode_window(out, q, k_cache, v_cache, block_tables, seq_lens, window, sinks, scale, out_lse,
//               stream)
PyObject* decode_window(PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  const at::Tensor *tq, *tk, *tb;
  if (!(tq = look(a[1], "q", kBf16, 3)) || !contiguous(*tq, "q") ||
      !(tk = look(a[2], "k_cache", kBf16, 4)) || !(tb = look(a[4], "block_tables", kI32, 2)))
    return nullptr;
  const Shape qs = tq->sizes(), ks = tk->sizes();
  const int dev = static_cast<int>(tq->get_device());
  const int64_t blocks = tb->size(1);
  int window, sinks;
  void *out, *k, *v, *bt, *sl, *lse, *stream;
  float scale;
  if (!tensor(a[2], "k_cache", kBf16, {ks[0], ks[1], ks[2], qs[2]}, dev, &k) ||
      !tensor(a[0], "out", kBf16, qs, dev, &out) ||
      !tensor(a[3], "v_cache", kBf16, ks, dev, &v) ||
      !tensor(a[4], "block_tables", kI32, {qs[0], blocks}, dev, &bt) ||
      !tensor(a[5], "seq_lens", kI32, {qs[0]}, dev, &sl) ||
      !whole(a[6], "window", 1, INT_MAX, &window) || !whole(a[7], "sinks", 0, INT_MAX, &sinks) ||
      !real(a[8], &scale) || !optional(a[9], "out_lse", kF32, {qs[0], qs[1]}, dev, &lse) ||
      !fits(qs[0], "q") || !fits(qs[1], "q") || !fits(qs[2], "q") ||
      !fits(blocks, "block_tables") || !fits(ks[1], "k_cache") || !fits(ks[2], "k_cache") ||
      !queue(a[10], dev, &stream))
    return nullptr;
  const void* q = tq->data_ptr();
  const int S = static_cast<int>(qs[0]), Hq = static_cast<int>(qs[1]), D = static_cast<int>(qs[2]),
            bs = static_cast<int>(ks[1]), Hkv = static_cast<int>(ks[2]);
  const int64_t nb = ks[0];
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pa_decode_window(out, q, k, v, static_cast<const int32_t*>(bt), static_cast<int>(blocks),
                        static_cast<const int32_t*>(sl), S, Hq, Hkv, D, bs, nb, window, sinks,
                        scale, static_cast<float*>(lse), stream);
  Py_END_ALLOW_THREADS;
  return done("pa_decode_window", rc);
}

// prefill_window(out, q, k_cache, v_cache, block_tables, cu_q_lens, q_start_pos, seq_lens,
//                max_q_len, window, sinks, scale, out_lse, stream)
PyObject* prefill_window(PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 14)) return nullptr;
  const at::Tensor *tq, *tk, *tb, *tc;
  if (!(tq = look(a[1], "q", kBf16, 3)) || !contiguous(*tq, "q") ||
      !(tk = look(a[2], "k_cache", kBf16, 4)) || !(tb = look(a[4], "block_tables", kI32, 2)) ||
      !(tc = look(a[5], "cu_q_lens", kI32, 1)))
    return nullptr;
  const Shape qs = tq->sizes(), ks = tk->sizes();
  const int dev = static_cast<int>(tq->get_device());
  const int64_t blocks = tb->size(1), chunks = tc->size(0) - 1;
  if (chunks < 0) {
    PyErr_SetString(PyExc_ValueError, "cu_q_lens must hold one more entry than there are chunks");
    return nullptr;
  }
  int max_q, window, sinks;
  void *out, *k, *v, *bt, *cu, *start, *sl, *lse, *stream;
  float scale;
  if (!tensor(a[2], "k_cache", kBf16, {ks[0], ks[1], ks[2], qs[2]}, dev, &k) ||
      !tensor(a[0], "out", kBf16, qs, dev, &out) ||
      !tensor(a[3], "v_cache", kBf16, ks, dev, &v) ||
      !tensor(a[4], "block_tables", kI32, {chunks, blocks}, dev, &bt) ||
      !tensor(a[5], "cu_q_lens", kI32, {chunks + 1}, dev, &cu) ||
      !tensor(a[6], "q_start_pos", kI32, {chunks}, dev, &start) ||
      !tensor(a[7], "seq_lens", kI32, {chunks}, dev, &sl) ||
      !whole(a[8], "max_q_len", 0, INT_MAX, &max_q) ||
      !whole(a[9], "window", 1, INT_MAX, &window) || !whole(a[10], "sinks", 0, INT_MAX, &sinks) ||
      !real(a[11], &scale) || !optional(a[12], "out_lse", kF32, {qs[0], qs[1]}, dev, &lse) ||
      !fits(qs[0], "q") || !fits(qs[1], "q") || !fits(qs[2], "q") ||
      !fits(blocks, "block_tables") || !fits(ks[1], "k_cache") || !fits(ks[2], "k_cache") ||
      !fits(chunks, "cu_q_lens") || !queue(a[13], dev, &stream))
    return nullptr;
  const void* q = tq->data_ptr();
  const int T = static_cast<int>(qs[0]), Hq = static_cast<int>(qs[1]), D = static_cast<int>(qs[2]),
            bs = static_cast<int>(ks[1]), Hkv = static_cast<int>(ks[2]);
  const int64_t nb = ks[0];
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = pa_prefill_window(out, q, k, v, static_cast<const int32_t*>(bt), static_cast<int>(blocks),
                         static_cast<const int32_t*>(cu), static_cast<const int32_t*>(start),
                         static_cast<const int32_t*>(sl), static_cast<int>(chunks), T, max_q, Hq,
                         Hkv, D, bs, nb, window, sinks, scale, static_cast<float*>(lse), stream);
  Py_END_ALLOW_THREADS;
  return done("pa_prefill_window", rc);
}

// norm_rope(q_out, k_out, q, k, v, positions, increments, k_cache, v_cache, slot_mapping,
//           k_scales, v_scales, q_weight, k_weight, eps, interleaved, rope_factor, stream, e4m3)
PyObject* norm_rope(PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 19)) return nullptr;
  const int fp8 = PyObject_IsTrue(a[18]), il = PyObject_IsTrue(a[15]);
  if (fp8 < 0 || il < 0) return nullptr;
  const at::Tensor *tq, *tk;
  if (!(tq = look(a[2], "q", kBf16, 3)) || !(tk = look(a[3], "k", kBf16, 3))) return nullptr;
  const Shape qs = tq->sizes();
  const int dev = static_cast<int>(tq->get_device());
  const int64_t T = qs[0], Hq = qs[1], Hkv = tk->size(1), D = qs[2];
  void *q_out, *k_out, *q, *k, *v = nullptr, *pos = nullptr, *inc = nullptr, *kc = nullptr,
                              *vc = nullptr, *slots = nullptr, *sk = nullptr, *sv = nullptr, *qw,
                              *kw, *stream;
  int64_t q_stride, k_stride, v_stride = 0, nb = 0, bs = 0, rot = 0;
  float eps, factor;
  if (!rows(*tq, "q", qs, dev, &q, &q_stride) ||
      !rows(*tk, "k", {T, Hkv, D}, dev, &k, &k_stride))
    return nullptr;
  if (fp8 || a[7] != Py_None || a[8] != Py_None) {
    const at::ScalarType type = fp8 ? kU8 : kBf16;
    const at::Tensor *tv, *tp;
    if (!(tv = look(a[4], "v", kBf16, 3)) || !rows(*tv, "v", {T, Hkv, D}, dev, &v, &v_stride) ||
        !(tp = look(a[7], "k_cache", type, 4)))
      return nullptr;
    nb = tp->size(0);
    bs = tp->size(1);
    if (!tensor(a[7], "k_cache", type, {nb, bs, Hkv, D}, dev, &kc) ||
        !tensor(a[8], "v_cache", type, {nb, bs, Hkv, D}, dev, &vc) ||
        !tensor(a[9], "slot_mapping", kI64, {T}, dev, &slots))
      return nullptr;
  }
  if (fp8 && (!tensor(a[10], "k_scales", kF32, {Hkv}, dev, &sk) ||
              !tensor(a[11], "v_scales", kF32, {Hkv}, dev, &sv)))
    return nullptr;
  if (a[6] != Py_None) {
    const at::Tensor* ti = look(a[6], "increments", kI64, 1);
    if (!ti || !tensor(a[6], "increments", kI64, {ti->size(0)}, dev, &inc) ||
        !tensor(a[5], "positions", kI64, {T}, dev, &pos))
      return nullptr;
    const int64_t pairs = ti->size(0);
    rot = 2 * (pairs < INT_MAX / 2 ? pairs : INT_MAX / 2);  // (a huge one is refused below)
  }
  if (!tensor(a[0], "q_out", kBf16, qs, dev, &q_out) ||
      !optional(a[1], "k_out", kBf16, {T, Hkv, D}, dev, &k_out) ||
      !optional(a[12], "q_weight", kF32, {D}, dev, &qw) ||
      !optional(a[13], "k_weight", kF32, {D}, dev, &kw) || !real(a[14], &eps) ||
      !real(a[16], &factor) || !fits(T, "q") || !fits(Hq, "q") || !fits(D, "q") ||
      !fits(Hkv, "k") || !fits(bs, "k_cache") || !queue(a[17], dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  if (fp8)
    rc = pa_qk_norm_rope_cache_fp8(
        q_out, k_out, q, k, v, q_stride, k_stride, v_stride, static_cast<float*>(qw),
        static_cast<float*>(kw), eps, static_cast<int64_t*>(pos), static_cast<int64_t*>(inc),
        static_cast<int>(rot), il, factor, kc, vc, static_cast<int64_t*>(slots),
        static_cast<float*>(sk), static_cast<float*>(sv), static_cast<int>(T),
        static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(D), static_cast<int>(bs), nb,
        stream);
  else
    rc = pa_qk_norm_rope_cache(
        q_out, k_out, q, k, v, q_stride, k_stride, v_stride, static_cast<float*>(qw),
        static_cast<float*>(kw), eps, static_cast<int64_t*>(pos), static_cast<int64_t*>(inc),
        static_cast<int>(rot), il, factor, kc, vc, static_cast<int64_t*>(slots),
        static_cast<int>(T), static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(D),
        static_cast<int>(bs), nb, stream);
  Py_END_ALLOW_THREADS;
  return done(fp8 ? "pa_qk_norm_rope_cache_fp8" : "pa_qk_norm_rope_cache", rc);
}

// No C++ exception (of a tensor without storage, say) leaves for the interpreter.
template <PyObject* (*f)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return f(a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// setup(the exception class of a refused call)
PyObject* setup(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XDECREF(g_error);
  g_error = error;
  Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction method(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"setup", setup, METH_O, nullptr},
    {"decode_window", method(guarded<decode_window>), METH_FASTCALL, nullptr},
    {"prefill_window", method(guarded<prefill_window>), METH_FASTCALL, nullptr},
    {"norm_rope", method(guarded<norm_rope>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycall(void) {
  if (!(n_stream = PyUnicode_InternFromString("cuda_stream"))) return nullptr;
  return PyModule_Create(&module);
}
