// Python's side of the attention calls: argument checks and marshalling for the C
// ABI, as a CPython extension (`_calls`).  Plain CPython: tensors are asked for
// their shape, strides and address by their own Python methods, nothing of torch is
// linked.  The kernels of a decode step take 4 to 10 us each, and the host's side of a
// call written in Python with ctypes took as long: calls queued back to back went
// from 10.0 to 6.5 us (kv_slots, 64 requests), 10.3 to 6.7 (qk_norm_rope, 64 tokens)
// and 9.5 to 7.0 (attn_prompt, 129 tokens).  A third of what is left is the outputs'
// allocation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <cstdint>

#include "moe_fp4.h"

namespace {

// set once by setup()
PyTypeObject* g_tensor;
PyObject *g_bf16, *g_i32, *g_f32, *g_u8, *g_raw_stream, *g_check, *g_describe, *g_current_stream, *g_under_stream, *g_get_device,
    *g_under_device;

struct Names {
  PyObject *dtype, *shape, *stride, *data_ptr, *get_device, *is_contiguous, *new_empty, *record_stream, *cuda_stream,
      *element_size, *numel, *split, *enter, *exit, *device_index;
} n_;

// An owned reference.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* x = nullptr) : p(x) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  void set(PyObject* x) {
    Py_XDECREF(p);
    p = x;
  }
  PyObject* give() {
    PyObject* x = p;
    p = nullptr;
    return x;
  }
};

bool given(PyObject* x) { return x && x != Py_None; }

// ---------------------------------------------------------------- arguments
constexpr int kMaxArgs = 16;

// Positional and keyword arguments into out[0 .. n), in the order of `names`.
bool parse(const char* fn, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames, PyObject* const* names, int n,
           int required, PyObject** out) {
  for (int i = 0; i < n; ++i) out[i] = nullptr;
  if (nargs > n) {
    PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments", fn, n);
    return false;
  }
  for (Py_ssize_t i = 0; i < nargs; ++i) out[i] = args[i];
  const Py_ssize_t kw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t k = 0; k < kw; ++k) {
    PyObject* name = PyTuple_GET_ITEM(kwnames, k);
    int at = -1;
    for (int i = 0; i < n && at < 0; ++i)
      if (names[i] == name) at = i;                                 // both interned, as a rule
    for (int i = 0; i < n && at < 0; ++i)
      if (PyUnicode_Compare(names[i], name) == 0) at = i;
    if (at < 0) {
      PyErr_Format(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", fn, name);
      return false;
    }
    if (out[at]) {
      PyErr_Format(PyExc_TypeError, "%s() got multiple values for argument '%U'", fn, name);
      return false;
    }
    out[at] = args[nargs + k];
  }
  for (int i = 0; i < required; ++i)
    if (!out[i]) {
      PyErr_Format(PyExc_TypeError, "%s() missing required argument '%U'", fn, names[i]);
      return false;
    }
  return true;
}

bool as_i64(PyObject* x, int64_t* v) {
  *v = PyLong_AsLongLong(x);
  return !(*v == -1 && PyErr_Occurred());
}
bool as_i32(PyObject* x, const char* name, int32_t* v) {
  int64_t w;
  if (!as_i64(x, &w)) return false;
  if (w < INT32_MIN || w > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s is no 32-bit number", name);
    return false;
  }
  *v = (int32_t)w;
  return true;
}
bool fits_i32(int64_t v, const char* name) {
  if (v <= INT32_MAX) return true;
  PyErr_Format(PyExc_ValueError, "%s: over 2^31 - 1", name);
  return false;
}
bool as_float(PyObject* x, float* v) {
  const double d = PyFloat_AsDouble(x);
  *v = (float)d;
  return !(d == -1.0 && PyErr_Occurred());
}

// ------------------------------------------------------------------ tensors
struct Shape {
  int64_t d[4];
};

bool is_tensor(PyObject* t) { return PyObject_TypeCheck(t, g_tensor); }

// Raises the ValueError that says what is wrong with the tensor.
bool describe(PyObject* t, const char* name, PyObject* dtype, int ndim, int index) {
  Ref r(PyObject_CallFunction(g_describe, "OsOii", t ? t : Py_None, name, dtype, ndim, index));
  return false;
}

bool has_dtype(PyObject* t, PyObject* dtype) {
  Ref d(PyObject_GetAttr(t, n_.dtype));
  if (!d.p) PyErr_Clear();
  return d.p == dtype;
}

// The device's index, -1 without one.
int device_of(PyObject* t) {
  Ref d(PyObject_CallMethodNoArgs(t, n_.get_device));
  const long v = d.p ? PyLong_AsLong(d.p) : -1;
  if (PyErr_Occurred()) PyErr_Clear();
  return (int)v;
}

bool gpu(PyObject* t, const char* name, int* index) {
  *index = is_tensor(t) ? device_of(t) : -1;
  if (*index >= 0) return true;
  PyErr_Format(PyExc_ValueError, "%s must be a GPU tensor", name);
  return false;
}

// The numbers of a tuple of `ndim`; false: another length.
bool numbers(PyObject* tuple, int ndim, int64_t* out) {
  if (!tuple || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != ndim) return false;
  for (int i = 0; i < ndim; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
  return true;
}
bool shape_of(PyObject* t, int ndim, Shape* s) {
  Ref r(PyObject_GetAttr(t, n_.shape));
  return numbers(r.p, ndim, s->d);
}
bool strides_of(PyObject* t, int ndim, Shape* s) {
  Ref r(PyObject_CallMethodNoArgs(t, n_.stride));
  return numbers(r.p, ndim, s->d);
}
bool address_of(PyObject* t, void** p) {
  Ref r(PyObject_CallMethodNoArgs(t, n_.data_ptr));
  *p = r.p ? (void*)(uintptr_t)PyLong_AsUnsignedLongLongMask(r.p) : nullptr;
  return r.p != nullptr;
}
bool contiguous(PyObject* t) {
  Ref r(PyObject_CallMethodNoArgs(t, n_.is_contiguous));
  return r.p == Py_True;
}

// Address and shape of a contiguous tensor.
bool flat(PyObject* t, const char* name, PyObject* dtype, int ndim, int index, void** p, Shape* s) {
  if (!t || !is_tensor(t) || !has_dtype(t, dtype) || device_of(t) != index || !shape_of(t, ndim, s) || !contiguous(t)) {
    if (!PyErr_Occurred()) describe(t, name, dtype, ndim, index);
    return false;
  }
  return address_of(t, p);
}

// Address, row stride and columns of an int32 table whose rows are contiguous.
bool table(PyObject* t, const char* name, int64_t rows, int index, void** p, int64_t* stride, int64_t* cols) {
  Shape s, st;
  if (!t || !is_tensor(t) || !has_dtype(t, g_i32) || device_of(t) != index || !shape_of(t, 2, &s) || !strides_of(t, 2, &st) ||
      (s.d[1] > 1 && st.d[1] != 1)) {
    if (!PyErr_Occurred()) describe(t, name, g_i32, 2, index);
    return false;
  }
  if (s.d[0] < rows) {
    PyErr_Format(PyExc_ValueError, "%s needs a row for each of %lld requests", name, (long long)rows);
    return false;
  }
  *stride = s.d[0] > 1 ? st.d[0] : s.d[1];
  *cols = s.d[1];
  return fits_i32(s.d[1], name) && address_of(t, p);
}

// bf16 [tokens, heads, dim], any token and head strides, dim contiguous; want: the
// sizes that it must have, -1 for any.
bool heads(PyObject* t, const char* name, int index, const Shape& want, moe_heads* out, Shape* s) {
  Shape st;
  if (!t || !is_tensor(t) || !has_dtype(t, g_bf16) || device_of(t) != index || !shape_of(t, 3, s) || !strides_of(t, 3, &st) ||
      (s->d[2] > 1 && st.d[2] != 1)) {
    if (!PyErr_Occurred()) describe(t, name, g_bf16, 3, index);
    return false;
  }
  for (int i = 0; i < 3; ++i)
    if (want.d[i] >= 0 && s->d[i] != want.d[i]) {
      PyErr_Format(PyExc_ValueError, "%s: shape (%lld, %lld, %lld) does not fit (tokens %lld, heads %lld, dim %lld; -1: any)",
                   name, (long long)s->d[0], (long long)s->d[1], (long long)s->d[2], (long long)want.d[0],
                   (long long)want.d[1], (long long)want.d[2]);
      return false;
    }
  // the strides of dimensions of one element say nothing
  out->head_stride = s->d[1] == 1 ? s->d[2] : st.d[1];
  out->token_stride = s->d[0] == 1 ? (s->d[1] - 1) * out->head_stride + s->d[2] : st.d[0];
  void* p;
  if (!fits_i32(s->d[1], name) || !fits_i32(s->d[2], name) || !address_of(t, &p)) return false;
  out->data = p;
  return true;
}

bool cache(PyObject* k, PyObject* v, int index, int64_t kv_heads, int64_t k_dim, moe_kv_cache* out, int64_t* v_dim) {
  Shape ks, vs;
  void *kp, *vp;
  if (!flat(k, "k_cache", g_bf16, 4, index, &kp, &ks) || !flat(v, "v_cache", g_bf16, 4, index, &vp, &vs)) return false;
  if ((kv_heads >= 0 && ks.d[2] != kv_heads) || ks.d[3] != k_dim || vs.d[0] != ks.d[0] || vs.d[1] != ks.d[1] ||
      vs.d[2] != ks.d[2]) {
    PyErr_Format(PyExc_ValueError, "k_cache %R / v_cache %R do not fit (pages, page_size, %lld heads, %lld)",
                 Ref(PyObject_GetAttr(k, n_.shape)).p, Ref(PyObject_GetAttr(v, n_.shape)).p,
                 (long long)(kv_heads >= 0 ? kv_heads : ks.d[2]), (long long)k_dim);
    return false;
  }
  if (!fits_i32(ks.d[1], "page_size") || !fits_i32(ks.d[2], "heads") || !fits_i32(vs.d[3], "v_dim")) return false;
  out->k = kp;
  out->v = vp;
  out->num_pages = ks.d[0];
  out->page_size = (int32_t)ks.d[1];
  *v_dim = vs.d[3];
  return true;
}

// like.new_empty(sizes[, dtype]); its address.
PyObject* make(PyObject* like, int ndim, const int64_t* d, PyObject* dtype, void** p) {
  Ref size(PyTuple_New(ndim));
  if (!size.p) return nullptr;
  for (int i = 0; i < ndim; ++i) PyTuple_SET_ITEM(size.p, i, PyLong_FromLongLong(d[i]));
  Ref t;
  if (dtype) {
    static PyObject* kw = Py_BuildValue("(s)", "dtype");
    PyObject* a[3] = {like, size.p, dtype};
    t.set(PyObject_VectorcallMethod(n_.new_empty, a, 2, kw));
  } else {
    PyObject* a[2] = {like, size.p};
    t.set(PyObject_VectorcallMethod(n_.new_empty, a, 2, nullptr));
  }
  if (!t.p || !address_of(t.p, p)) return nullptr;
  return t.give();
}

// The arguments' device is the current one while the call runs (every device's default
// stream has the same handle: launched from another device it would be that one's).
// A stream that the caller names is the current one while the call makes its tensors:
// their memory is then free in that stream's own order.  (A block from another
// stream's pool may still be written by what is queued there.)  The outputs are made
// known to the stream that was current before, where the caller may read them.
class Placed {
 public:
  ~Placed() {
    if (context_) {
      PyObject *type, *value, *trace;
      PyErr_Fetch(&type, &value, &trace);
      PyObject* a[4] = {context_, Py_None, Py_None, Py_None};
      Ref r(PyObject_VectorcallMethod(n_.exit, a, 4, nullptr));
      if (!r.p) PyErr_WriteUnraisable(context_);
      PyErr_Restore(type, value, trace);
      Py_DECREF(context_);
    }
    Py_XDECREF(outer_);
  }
  bool enter(PyObject* stream, int index) {
    Ref i(nullptr), c(nullptr);
    if (!given(stream)) {
      Ref now(PyObject_CallNoArgs(g_get_device));
      const long at = now.p ? PyLong_AsLong(now.p) : -1;
      if (at == index || PyErr_Occurred()) return !PyErr_Occurred();
      i.set(PyLong_FromLong(index));
      c.set(i.p ? PyObject_CallOneArg(g_under_device, i.p) : nullptr);
    } else {
      Ref of(PyObject_GetAttr(stream, n_.device_index));
      const long at = of.p ? PyLong_AsLong(of.p) : -1;
      if (PyErr_Occurred()) return false;
      if (at != index) {
        PyErr_Format(PyExc_ValueError, "stream of cuda:%ld, the arguments are on cuda:%d", at, index);
        return false;
      }
      i.set(PyLong_FromLong(index));
      outer_ = i.p ? PyObject_CallOneArg(g_current_stream, i.p) : nullptr;
      c.set(outer_ ? PyObject_CallOneArg(g_under_stream, stream) : nullptr);
    }
    Ref r(c.p ? PyObject_CallMethodNoArgs(c.p, n_.enter) : nullptr);
    if (!r.p) return false;
    context_ = c.give();
    return true;
  }
  bool known(PyObject* const* made, int n) const {
    for (int k = 0; k < n && outer_; ++k) {
      if (!made[k]) continue;
      PyObject* a[2] = {made[k], outer_};
      Ref r(PyObject_VectorcallMethod(n_.record_stream, a, 2, nullptr));
      if (!r.p) return false;
    }
    return true;
  }

 private:
  PyObject *context_ = nullptr, *outer_ = nullptr;
};

// The stream to launch on.
bool stream_of(PyObject* stream, int index, hipStream_t* out) {
  Ref i(given(stream) ? nullptr : PyLong_FromLong(index));
  Ref s(given(stream) ? PyObject_GetAttr(stream, n_.cuda_stream) : (i.p ? PyObject_CallOneArg(g_raw_stream, i.p) : nullptr));
  if (!s.p) return false;
  *out = (hipStream_t)(uintptr_t)PyLong_AsUnsignedLongLongMask(s.p);
  return !PyErr_Occurred();
}

bool check(moe_status st, const char* fn) {
  if (st == MOE_OK) return true;
  Ref r(PyObject_CallFunction(g_check, "is", (int)st, fn));
  if (r.p) PyErr_Format(PyExc_RuntimeError, "%s: status %d", fn, (int)st);
  return false;
}

// A workspace that was given, or of `need` bytes made here.
bool workspace(PyObject* given_ws, PyObject* like, int index, size_t need, Ref* made, void** p, size_t* bytes) {
  *p = nullptr;
  *bytes = 0;
  if (!given(given_ws)) {
    if (need == 0) return true;
    const int64_t d = (int64_t)need;
    made->set(make(like, 1, &d, g_u8, p));
    *bytes = need;
    return made->p != nullptr;
  }
  if (!is_tensor(given_ws) || device_of(given_ws) != index || !contiguous(given_ws)) {
    PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous GPU tensor");
    return false;
  }
  Ref a(PyObject_CallMethodNoArgs(given_ws, n_.numel)), b(PyObject_CallMethodNoArgs(given_ws, n_.element_size));
  if (!a.p || !b.p) return false;
  *bytes = (size_t)PyLong_AsLongLong(a.p) * (size_t)PyLong_AsLongLong(b.p);
  return !PyErr_Occurred() && address_of(given_ws, p);
}

// An output that was given, checked, or made: bf16 [T, H, D].
bool output_heads(PyObject* t, const char* name, PyObject* like, int index, int64_t T, int64_t H, int64_t D, Ref* made,
                  PyObject** out, moe_heads* h) {
  if (given(t)) {
    Shape s;
    *out = t;
    return heads(t, name, index, Shape{{T, H, D, 0}}, h, &s);
  }
  const int64_t d[3] = {T, H, D};
  void* p;
  made->set(make(like, 3, d, nullptr, &p));
  if (!made->p) return false;
  *out = made->p;
  *h = moe_heads{p, H * D, D};
  return true;
}

// lse: given, wanted (made) or absent (None).
bool output_lse(PyObject* t, PyObject* want, PyObject* like, int index, int64_t T, int64_t H, Ref* made, PyObject** out,
                void** p) {
  *p = nullptr;
  *out = Py_None;
  if (given(t)) {
    Shape s;
    if (!flat(t, "lse", g_f32, 2, index, p, &s)) return false;
    if (s.d[0] != T || s.d[1] != H) {
      PyErr_Format(PyExc_ValueError, "lse must be (%lld, %lld)", (long long)T, (long long)H);
      return false;
    }
    *out = t;
    return true;
  }
  const int yes = want ? PyObject_IsTrue(want) : 0;
  if (yes <= 0) return yes == 0;
  const int64_t d[2] = {T, H};
  made->set(make(like, 2, d, g_f32, p));
  *out = made->p;
  return made->p != nullptr;
}

bool scale_of(PyObject* x, int64_t k_dim, float* scale) {
  if (given(x)) return as_float(x, scale);
  *scale = (float)(1.0 / std::sqrt((double)k_dim));
  return true;
}

// -------------------------------------------------------------------- calls
#define NAMES(...)                                                             \
  static const char* const words[] = {__VA_ARGS__};                           \
  constexpr int N = sizeof(words) / sizeof(words[0]);                          \
  static_assert(N <= kMaxArgs, "");                                            \
  static PyObject* names[N];                                                   \
  if (!names[N - 1])                                                           \
    for (int i = 0; i < N; ++i) names[i] = PyUnicode_InternFromString(words[i]); \
  PyObject* a[N]

PyObject* kv_slots(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  NAMES("cached_lens", "new_lens", "free_pages", "block_table", "page_size", "max_new", "position_base", "slots",
        "positions", "cu_new", "counts", "stream");
  if (!parse("kv_slots", args, nargs, kwnames, names, N, 6, a)) return nullptr;
  int dev;
  Placed placed;
  void *cached, *fresh, *pool, *tab, *p[4];
  Shape cs, ns, fs;
  int64_t stride, blocks, most;
  int32_t page, base = 0;
  if (!gpu(a[0], "cached_lens", &dev) || !placed.enter(a[11], dev) || !flat(a[0], "cached_lens", g_i32, 1, dev, &cached, &cs) ||
      !flat(a[1], "new_lens", g_i32, 1, dev, &fresh, &ns) || !flat(a[2], "free_pages", g_i32, 1, dev, &pool, &fs))
    return nullptr;
  const int64_t B = cs.d[0];
  if (ns.d[0] != B) {
    PyErr_SetString(PyExc_ValueError, "cached_lens and new_lens must have an entry for each request");
    return nullptr;
  }
  if (!fits_i32(B, "cached_lens") || !table(a[3], "block_table", B, dev, &tab, &stride, &blocks) ||
      !as_i32(a[4], "page_size", &page) || !as_i64(a[5], &most) || (a[6] && !as_i32(a[6], "position_base", &base)))
    return nullptr;
  Ref made[4], pieces;
  PyObject *out[4], *own[4];
  const int64_t size[4] = {most < 0 ? 0 : most, most < 0 ? 0 : most, B + 1, 3};
  const bool all = !given(a[7]) && !given(a[8]) && !given(a[9]) && !given(a[10]);
  if (all) {
    // one allocation in four pieces takes 2/3 of the time of four
    const int64_t total = size[0] + size[1] + size[2] + size[3];
    void* base;
    made[0].set(make(a[0], 1, &total, nullptr, &base));
    if (!made[0].p) return nullptr;
    Ref sizes(Py_BuildValue("(LLLL)", (long long)size[0], (long long)size[1], (long long)size[2], (long long)size[3]));
    PyObject* v[2] = {made[0].p, sizes.p};
    pieces.set(sizes.p ? PyObject_VectorcallMethod(n_.split, v, 2, nullptr) : nullptr);
    if (pieces.p) pieces.set(PySequence_Tuple(pieces.p));
    if (!pieces.p || PyTuple_GET_SIZE(pieces.p) != 4) return nullptr;
    int64_t before = 0;
    for (int i = 0; i < 4; ++i) {
      out[i] = PyTuple_GET_ITEM(pieces.p, i);
      p[i] = (int32_t*)base + before;
      before += size[i];
      own[i] = i == 0 ? made[0].p : nullptr;
    }
  }
  for (int i = 0; i < 4 && !all; ++i) {
    PyObject* t = a[7 + i];
    if (given(t)) {
      Shape s;
      if (!flat(t, words[7 + i], g_i32, 1, dev, &p[i], &s)) return nullptr;
      if (s.d[0] < size[i]) {
        PyErr_Format(PyExc_ValueError, "%s needs %lld elements", words[7 + i], (long long)size[i]);
        return nullptr;
      }
      out[i] = t;
    } else {
      made[i].set(make(a[0], 1, &size[i], nullptr, &p[i]));
      if (!made[i].p) return nullptr;
      out[i] = made[i].p;
    }
    own[i] = made[i].p;
  }
  hipStream_t stream;
  if (!stream_of(a[11], dev, &stream) || !placed.known(own, 4)) return nullptr;
  if (!check(moe_kv_slots((const int32_t*)cached, (const int32_t*)fresh, (int32_t)B, (const int32_t*)pool, fs.d[0], page,
                          (int32_t*)tab, stride, (int32_t)blocks, base, most, (int32_t*)p[0], (int32_t*)p[1],
                          (int32_t*)p[2], (int32_t*)p[3], stream),
             "moe_kv_slots"))
    return nullptr;
  return all ? pieces.give() : PyTuple_Pack(4, out[0], out[1], out[2], out[3]);
}

PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  NAMES("q", "k", "positions", "cos_sin", "q_weight", "k_weight", "eps", "interleaved", "v", "k_cache", "v_cache", "slots",
        "want_k", "q_out", "k_out", "stream");
  if (!parse("qk_norm_rope", args, nargs, kwnames, names, N, 4, a)) return nullptr;
  int dev;
  Placed placed;
  moe_heads hq, hk, hv, ho, hko;
  Shape qs, ks, s;
  if (!gpu(a[0], "q", &dev) || !placed.enter(a[15], dev) || !heads(a[0], "q", dev, Shape{{-1, -1, -1, 0}}, &hq, &qs)) return nullptr;
  const int64_t T = qs.d[0], D = qs.d[2];
  if (!heads(a[1], "k", dev, Shape{{T, -1, D, 0}}, &hk, &ks)) return nullptr;
  const int64_t Hkv = ks.d[1];
  moe_rope_params prm = {(int32_t)qs.d[1], (int32_t)Hkv, (int32_t)D, 0, 0, 0, 0, 1e-6f};
  void *pos = nullptr, *cs = nullptr, *w[2] = {nullptr, nullptr}, *slots = nullptr;
  if (given(a[3])) {
    Shape c;
    if (!flat(a[3], "cos_sin", g_f32, 2, dev, &cs, &c) || !flat(a[2], "positions", g_i32, 1, dev, &pos, &s)) return nullptr;
    if (s.d[0] < T) {
      PyErr_SetString(PyExc_ValueError, "positions needs an entry for each token");
      return nullptr;
    }
    if (!fits_i32(c.d[0], "cos_sin") || !fits_i32(c.d[1], "cos_sin")) return nullptr;
    prm.max_position = (int32_t)c.d[0];
    prm.rot_dim = (int32_t)c.d[1];
  }
  for (int i = 0; i < 2; ++i) {
    if (!given(a[4 + i])) continue;
    if (!flat(a[4 + i], words[4 + i], g_f32, 1, dev, &w[i], &s)) return nullptr;
    if (s.d[0] != D) {
      PyErr_Format(PyExc_ValueError, "q_weight and k_weight need %lld elements", (long long)D);
      return nullptr;
    }
  }
  if (a[6] && !as_float(a[6], &prm.eps)) return nullptr;
  if (a[7]) {
    prm.interleaved = PyObject_IsTrue(a[7]);
    if (prm.interleaved < 0) return nullptr;
  }
  moe_kv_cache c;
  const bool cached = given(a[9]);
  if (cached) {
    int64_t v_dim;
    if (!cache(a[9], a[10], dev, Hkv, D, &c, &v_dim) || !heads(a[8], "v", dev, Shape{{T, Hkv, v_dim, 0}}, &hv, &s) ||
        !flat(a[11], "slots", g_i32, 1, dev, &slots, &s))
      return nullptr;
    if (s.d[0] < T) {
      PyErr_SetString(PyExc_ValueError, "slots needs an entry for each token");
      return nullptr;
    }
    prm.v_dim = (int32_t)v_dim;
  }
  const int keep = a[12] ? PyObject_IsTrue(a[12]) : 1;
  if (keep < 0) return nullptr;
  Ref mq, mk;
  PyObject *q_out, *k_out = Py_None;
  if (!output_heads(a[13], "q_out", a[0], dev, T, qs.d[1], D, &mq, &q_out, &ho)) return nullptr;
  const bool write_k = given(a[14]) || keep;
  if (write_k && !output_heads(a[14], "k_out", a[1], dev, T, Hkv, D, &mk, &k_out, &hko)) return nullptr;
  PyObject* own[2] = {mq.p, mk.p};
  hipStream_t stream;
  if (!stream_of(a[15], dev, &stream) || !placed.known(own, 2)) return nullptr;
  if (!check(moe_qk_norm_rope(&hq, &hk, cached ? &hv : nullptr, T, &prm, (const int32_t*)pos, (const float*)cs,
                              (const float*)w[0], (const float*)w[1], &ho, write_k ? &hko : nullptr, cached ? &c : nullptr,
                              (const int32_t*)slots, stream),
             "moe_qk_norm_rope"))
    return nullptr;
  return PyTuple_Pack(2, q_out, k_out);
}

PyObject* attn_prompt(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  NAMES("q", "k", "v", "cu_q", "cu_k", "scale", "out", "lse", "want_lse", "workspace", "stream");
  if (!parse("attn_prompt", args, nargs, kwnames, names, N, 4, a)) return nullptr;
  int dev;
  Placed placed;
  moe_heads hq, hk, hv, ho;
  Shape qs, ks, vs, cq, ck;
  void *pq, *pk, *pl, *ws;
  if (!gpu(a[0], "q", &dev) || !placed.enter(a[10], dev) || !heads(a[0], "q", dev, Shape{{-1, -1, -1, 0}}, &hq, &qs) ||
      !heads(a[1], "k", dev, Shape{{-1, -1, qs.d[2], 0}}, &hk, &ks) ||
      !heads(a[2], "v", dev, Shape{{ks.d[0], ks.d[1], -1, 0}}, &hv, &vs) || !flat(a[3], "cu_q", g_i32, 1, dev, &pq, &cq))
    return nullptr;
  pk = pq;
  ck = cq;
  if (given(a[4]) && !flat(a[4], "cu_k", g_i32, 1, dev, &pk, &ck)) return nullptr;
  if (cq.d[0] < 1 || ck.d[0] != cq.d[0]) {
    PyErr_SetString(PyExc_ValueError, "cu_q and cu_k must have an entry for each sequence and the end");
    return nullptr;
  }
  const int64_t T = qs.d[0], H = qs.d[1], seqs = cq.d[0] - 1;
  moe_attn_params prm = {(int32_t)H, (int32_t)ks.d[1], (int32_t)qs.d[2], (int32_t)vs.d[2], 0.0f};
  size_t bytes;
  Ref mw, mo, ml;
  PyObject *out, *lse;
  if (!fits_i32(cq.d[0], "cu_q") || !scale_of(a[5], qs.d[2], &prm.scale) ||
      !workspace(a[9], a[0], dev, moe_attn_prompt_workspace_bytes((int32_t)seqs, T, ks.d[0], &prm), &mw, &ws, &bytes) ||
      !output_heads(a[6], "out", a[0], dev, T, H, vs.d[2], &mo, &out, &ho) ||
      !output_lse(a[7], a[8], a[0], dev, T, H, &ml, &lse, &pl))
    return nullptr;
  PyObject* own[2] = {mo.p, ml.p};
  hipStream_t stream;
  if (!stream_of(a[10], dev, &stream) || !placed.known(own, 2)) return nullptr;
  if (!check(moe_attn_prompt(&hq, &hk, &hv, (const int32_t*)pq, (const int32_t*)pk, (int32_t)seqs, T, ks.d[0], &prm, &ho,
                             (float*)pl, ws, bytes, stream),
             "moe_attn_prompt"))
    return nullptr;
  return PyTuple_Pack(2, out, lse);
}

PyObject* attn_decode(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  NAMES("q", "k_cache", "v_cache", "block_table", "lens", "max_len", "prefix_table", "prefix_len", "scale", "workspace",
        "out", "lse", "want_lse", "stream");
  if (!parse("attn_decode", args, nargs, kwnames, names, N, 6, a)) return nullptr;
  int dev;
  Placed placed;
  moe_heads hq, ho;
  moe_kv_cache c;
  Shape qs, s;
  void *tab, *lens, *prefix = nullptr, *pl, *ws;
  int64_t stride, blocks, most, prefix_blocks = 0, prefix_len = 0, v_dim;
  if (!gpu(a[0], "q", &dev) || !placed.enter(a[13], dev) || !heads(a[0], "q", dev, Shape{{-1, -1, -1, 0}}, &hq, &qs))
    return nullptr;
  const int64_t B = qs.d[0], H = qs.d[1];
  Shape ks;
  if (!cache(a[1], a[2], dev, -1, qs.d[2], &c, &v_dim) || !shape_of(a[1], 4, &ks) ||
      !table(a[3], "block_table", B, dev, &tab, &stride, &blocks) || !flat(a[4], "lens", g_i32, 1, dev, &lens, &s))
    return nullptr;
  if (s.d[0] < B) {
    PyErr_SetString(PyExc_ValueError, "lens needs an entry for each request");
    return nullptr;
  }
  if (given(a[6])) {
    if (!flat(a[6], "prefix_table", g_i32, 1, dev, &prefix, &s) || !fits_i32(s.d[0], "prefix_table")) return nullptr;
    prefix_blocks = s.d[0];
  }
  moe_attn_params prm = {(int32_t)H, (int32_t)ks.d[2], (int32_t)qs.d[2], (int32_t)v_dim, 0.0f};
  size_t bytes;
  Ref mw, mo, ml;
  PyObject *out, *lse;
  if (!fits_i32(B, "q") || !as_i64(a[5], &most) || (a[7] && !as_i64(a[7], &prefix_len)) || !scale_of(a[8], qs.d[2], &prm.scale) ||
      !workspace(a[9], a[0], dev, moe_attn_decode_workspace_bytes((int32_t)B, prefix_len, most, &prm), &mw, &ws, &bytes) ||
      !output_heads(a[10], "out", a[0], dev, B, H, v_dim, &mo, &out, &ho) ||
      !output_lse(a[11], a[12], a[0], dev, B, H, &ml, &lse, &pl))
    return nullptr;
  PyObject* own[2] = {mo.p, ml.p};
  hipStream_t stream;
  if (!stream_of(a[13], dev, &stream) || !placed.known(own, 2)) return nullptr;
  if (!check(moe_attn_decode(&hq, &c, (const int32_t*)tab, stride, (int32_t)blocks, (const int32_t*)lens, (int32_t)B, most,
                             (const int32_t*)prefix, (int32_t)prefix_blocks, prefix_len, &prm, &ho, (float*)pl, ws, bytes,
                             stream),
             "moe_attn_decode"))
    return nullptr;
  return PyTuple_Pack(2, out, lse);
}

PyObject* setup(PyObject*, PyObject* args) {
  PyObject *tensor, *bf16, *i32, *f32, *u8, *raw, *chk, *desc, *current, *under, *get, *device;
  if (!PyArg_ParseTuple(args, "OOOOOOOOOOOO", &tensor, &bf16, &i32, &f32, &u8, &raw, &chk, &desc, &current, &under, &get, &device))
    return nullptr;
  if (!PyType_Check(tensor)) {
    PyErr_SetString(PyExc_TypeError, "the tensor type is no type");
    return nullptr;
  }
  for (PyObject* x : {tensor, bf16, i32, f32, u8, raw, chk, desc, current, under, get, device}) Py_INCREF(x);   // for good
  g_tensor = (PyTypeObject*)tensor;
  g_bf16 = bf16;
  g_i32 = i32;
  g_f32 = f32;
  g_u8 = u8;
  g_raw_stream = raw;
  g_check = chk;
  g_describe = desc;
  g_current_stream = current;
  g_under_stream = under;
  g_get_device = get;
  g_under_device = device;
  Py_RETURN_NONE;
}

#define CALL(name, doc) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL | METH_KEYWORDS, doc}
#define STREAM_DOC                                                                                             \
  "``stream``: where the call runs, the current stream if None.  It has to come after what makes the arguments;\n" \
  "new outputs are made on it, and a reader on another stream has to wait for it."
PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "Names what the calls need of torch and of the package."},
    CALL(kv_slots,
         "kv_slots(cached_lens, new_lens, free_pages, block_table, page_size, max_new, position_base=0, slots=None, "
         "positions=None, cu_new=None, counts=None, stream=None)\n--\n\n"
         "Cache slots of a step's new tokens.  int32 tensors: cached_lens, new_lens [B], free_pages [F], block_table\n"
         "[B, blocks] (new pages are entered in place).  -> (slots [max_new], positions [max_new], cu_new [B + 1],\n"
         "counts [3]: pages taken, pages needed, tokens without a slot).  ``position_base``: length of a shared prefix.\n"
         STREAM_DOC),
    CALL(qk_norm_rope,
         "qk_norm_rope(q, k, positions, cos_sin, q_weight=None, k_weight=None, eps=1e-06, interleaved=False, v=None, "
         "k_cache=None, v_cache=None, slots=None, want_k=True, q_out=None, k_out=None, stream=None)\n--\n\n"
         "RMS norm of each head of q [T, Hq, D] and k [T, Hkv, D] (weights float32 [D]; None: no norm), the rotation by\n"
         "``cos_sin`` float32 [positions, rot_dim] (cosines, then sines; None: no rotation), and with a cache the write of\n"
         "the finished keys and of v [T, Hkv, Dv] to its rows ``slots``.  -> (q_out, k_out); k_out is None with\n"
         "``want_k=False`` (cache only).  q_out / k_out may be q / k.\n" STREAM_DOC),
    CALL(attn_prompt,
         "attn_prompt(q, k, v, cu_q, cu_k=None, scale=None, out=None, lse=None, want_lse=False, workspace=None, "
         "stream=None)\n--\n\n"
         "Causal attention over packed prompts: q [Tq, Hq, D], k [Tk, Hkv, D], v [Tk, Hkv, Dv], offsets cu_q, cu_k int32\n"
         "[B + 1] (cu_k None: cu_q).  Query i of a sequence sees keys 0 .. i + Lk - Lq.  -> (out [Tq, Hq, Dv], lse float32\n"
         "[Tq, Hq] or None).  Rows outside the offsets' ranges are not written.\n" STREAM_DOC),
    CALL(attn_decode,
         "attn_decode(q, k_cache, v_cache, block_table, lens, max_len, prefix_table=None, prefix_len=0, scale=None, "
         "workspace=None, out=None, lse=None, want_lse=False, stream=None)\n--\n\n"
         "One query per request, q [B, Hq, D], over the paged cache: the shared prefix (``prefix_len`` keys in the pages\n"
         "``prefix_table``), then the request's own ``lens`` keys in its ``block_table`` pages (int32).  ``max_len``: a\n"
         "longest own length known on the host.  -> (out [B, Hq, Dv], lse float32 [B, Hq] or None).\n" STREAM_DOC),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Argument checks and marshalling of the attention calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  auto name = [](PyObject** p, const char* s) { return (*p = PyUnicode_InternFromString(s)) != nullptr; };
  if (!name(&n_.dtype, "dtype") || !name(&n_.shape, "shape") || !name(&n_.stride, "stride") ||
      !name(&n_.data_ptr, "data_ptr") || !name(&n_.get_device, "get_device") || !name(&n_.is_contiguous, "is_contiguous") ||
      !name(&n_.new_empty, "new_empty") || !name(&n_.record_stream, "record_stream") ||
      !name(&n_.cuda_stream, "cuda_stream") || !name(&n_.element_size, "element_size") || !name(&n_.numel, "numel") || !name(&n_.split, "unsafe_split_with_sizes") ||
      !name(&n_.enter, "__enter__") || !name(&n_.exit, "__exit__") || !name(&n_.device_index, "device_index"))
    return nullptr;
  return PyModule_Create(&module);
}
