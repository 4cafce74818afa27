// Marshalling of the decode-step calls (CPython C API).  These calls put a few
// microseconds of work on the GPU, and asking five to nine tensors for type, shape,
// place and address from Python costs as much again.  Each function here asks the same
// questions of a call that is right in every respect, calls the C entry, and returns its
// status; for any other call it returns None, has called nothing, and the caller takes
// the Python path, which says what is wrong (or changes the device).
// (Time per call from Python: kq_gemv 8.4 to 4.5 us, the attention of short sequences 9.2
// to 4.9, page copies 6.4 to 3.4; a launch alone takes about 2.9.  Since then the caches'
// arrays are asked again at every call: 1.4 us more for a pair of caches.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>
#include <stdint.h>

#include "kq.h"

static PyObject *n_dtype, *n_shape, *n_get_device, *n_is_contiguous, *n_data_ptr, *n_cuda_stream,
    *n_view;
// what init() was given
static PyObject *t_bf16, *t_f32, *t_f16, *t_u8, *t_i8, *t_i32, *f_stream, *f_device;
static __typeof__(&kq_gemv) c_gemv;
static __typeof__(&kq_attn_decode_int4_kv) c_attn;
static __typeof__(&kq_kv_copy_pages) c_copy;

// A call that is not answered here: None, whatever was raised on the way.
static PyObject* other_path(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

static int as_int64(PyObject* o, int64_t* v) {
  if (!o || !PyLong_Check(o)) return 0;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return !over && !(*v == -1 && PyErr_Occurred());
}
static int as_int(PyObject* o, int* v) {
  int64_t w;
  if (!as_int64(o, &w) || w < INT_MIN || w > INT_MAX) return 0;
  *v = (int)w;
  return 1;
}

// The tensor's shape, when it has nd dimensions.
static int shape_of(PyObject* t, int nd, int64_t* shape) {
  PyObject* s = PyObject_GetAttr(t, n_shape);
  int ok = s && PyTuple_Check(s) && PyTuple_GET_SIZE(s) == nd;
  for (int i = 0; ok && i < nd; ++i) ok = as_int64(PyTuple_GET_ITEM(s, i), shape + i);
  Py_XDECREF(s);
  return ok;
}
static int device_of(PyObject* t, int64_t* at) {
  PyObject* d = PyObject_CallMethodNoArgs(t, n_get_device);
  const int ok = as_int64(d, at);
  Py_XDECREF(d);
  return ok;
}
static int has_dtype(PyObject* t, PyObject* dtype) {
  PyObject* d = PyObject_GetAttr(t, n_dtype);
  Py_XDECREF(d);                        // types of tensors are kept by their module
  return d == dtype;
}
static int address(PyObject* t, void** p) {
  PyObject* a = PyObject_CallMethodNoArgs(t, n_data_ptr);
  const int ok = a && PyLong_Check(a);
  if (ok) *p = PyLong_AsVoidPtr(a);
  Py_XDECREF(a);
  return ok && !PyErr_Occurred();
}
// Its address, when it is contiguous and on device `at`.
static int placed(PyObject* t, int64_t at, void** p) {
  int64_t d;
  if (!device_of(t, &d) || d != at) return 0;
  PyObject* c = PyObject_CallMethodNoArgs(t, n_is_contiguous);
  Py_XDECREF(c);                        // True or False
  return c == Py_True && address(t, p);
}
// ... and of this type and shape.
static int want(PyObject* t, PyObject* dtype, int nd, const int64_t* shape, int64_t at, void** p) {
  int64_t s[3];
  if (!has_dtype(t, dtype) || !shape_of(t, nd, s)) return 0;
  for (int i = 0; i < nd; ++i)
    if (s[i] != shape[i]) return 0;
  return placed(t, at, p);
}
static int float_type(PyObject* t, int* code) {
  PyObject* d = PyObject_GetAttr(t, n_dtype);
  Py_XDECREF(d);
  *code = d == t_bf16 ? KQ_BF16 : KQ_F32;
  return d && (d == t_bf16 || d == t_f32);
}

// The stream of a call on device `at`, when that is the current device.
static int stream_of(PyObject* given, int64_t at, void** stream) {
  PyObject* now = PyObject_CallNoArgs(f_device);
  int64_t d;
  const int here = as_int64(now, &d) && d == at;
  PyObject* s = NULL;
  if (here) {
    if (given == Py_None) s = PyObject_CallOneArg(f_stream, now);
    else if (PyLong_Check(given)) s = Py_NewRef(given);
    else s = PyObject_GetAttr(given, n_cuda_stream);
  }
  const int ok = s && PyLong_Check(s);
  if (ok) *stream = PyLong_AsVoidPtr(s);
  Py_XDECREF(s);
  Py_XDECREF(now);
  return ok && !PyErr_Occurred();
}

// gemv(fmt, x, codes, scales, zeros, tensor_scale, group, y, stream)
static PyObject* gemv(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  int fmt, group, xt, yt;
  int64_t xs[2], cs[2], at;
  void *x, *codes, *scales, *zeros = NULL, *tscale = NULL, *y, *stream;
  if (n_args != 9 || !c_gemv || !as_int(a[0], &fmt) || !as_int(a[6], &group) ||
      !shape_of(a[1], 2, xs) || !shape_of(a[2], 2, cs) || !device_of(a[1], &at) || at < 0)
    return other_path();
  const int64_t m = xs[0], k = xs[1], n = cs[0];
  const int64_t codes_shape[2] = {n, k / 2}, y_shape[2] = {m, n};
  if (k > INT_MAX) return other_path();
  int64_t s[2] = {n, 0}, one = 1;
  int ok = 0;
  switch (fmt) {
    case KQ_FMT_INT4_ASYM:
      s[1] = k / 128;
      ok = want(a[3], t_f16, 2, s, at, &scales) && want(a[4], t_f16, 2, s, at, &zeros);
      break;
    case KQ_FMT_INT4_SYM: ok = want(a[3], t_f32, 1, s, at, &scales); break;
    case KQ_FMT_NVFP4:
      s[1] = k / 16;
      ok = want(a[3], t_u8, 2, s, at, &scales) && want(a[5], t_f32, 1, &one, at, &tscale);
      break;
    case KQ_FMT_MXFP4:
      s[1] = k / 32;
      ok = want(a[3], t_u8, 2, s, at, &scales);
      break;
  }
  if (!ok || !float_type(a[1], &xt) || !placed(a[1], at, &x) ||
      !want(a[2], t_u8, 2, codes_shape, at, &codes) || !float_type(a[7], &yt) ||
      !want(a[7], yt == KQ_BF16 ? t_bf16 : t_f32, 2, y_shape, at, &y) ||
      !stream_of(a[8], at, &stream))
    return other_path();
  kq_status st;
  Py_BEGIN_ALLOW_THREADS
  st = c_gemv(fmt, x, xt, m, codes, scales, zeros, tscale, n, (int)k, group, y, yt, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// What a cache keeps of itself: (codes, scales, zeros, layers, num_slots, dim, index,
// layered).  The arrays are asked again at every call: they are the caller's, who may have
// resized them or exchanged their memory since (0.7 us a cache).
typedef struct {
  void* p[3];
  int64_t layers, slots, dim, at;
  int layered;
} Cache;
static int cache_of(PyObject* o, Cache* c) {
  PyObject* v = PyObject_GetAttr(o, n_view);
  int ok = v && PyTuple_CheckExact(v) && PyTuple_GET_SIZE(v) == 8 &&
           as_int64(PyTuple_GET_ITEM(v, 3), &c->layers) &&
           as_int64(PyTuple_GET_ITEM(v, 4), &c->slots) && as_int64(PyTuple_GET_ITEM(v, 5), &c->dim) &&
           as_int64(PyTuple_GET_ITEM(v, 6), &c->at) && c->dim <= INT_MAX && c->layers <= INT_MAX &&
           c->at >= 0;
  if (ok) {
    c->layered = PyTuple_GET_ITEM(v, 7) == Py_True;
    int64_t shape[3] = {c->layers, c->slots, c->dim / 2};
    const int skip = c->layered ? 0 : 1;
    ok = want(PyTuple_GET_ITEM(v, 0), t_u8, 3 - skip, shape + skip, c->at, &c->p[0]);
    shape[2] = c->dim / 128;
    for (int i = 1; ok && i < 3; ++i)
      ok = want(PyTuple_GET_ITEM(v, i), t_f16, 3 - skip, shape + skip, c->at, &c->p[i]);
  }
  Py_XDECREF(v);
  return ok;
}

// attn(q, k_cache, v_cache, k_signs, v_signs, block_table, page_size, seq_lens,
//      softmax_scale, out, workspace, window, sinks, stream)
static PyObject* attn(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  Cache k, v;
  int page, window, sinks;
  int64_t qs[3], ts[2], ws, at;
  void *q, *ksg = NULL, *vsg = NULL, *table, *lens, *out, *work, *stream;
  if (n_args != 14 || !c_attn || !cache_of(a[1], &k) || !cache_of(a[2], &v) ||
      !as_int(a[6], &page) || !as_int(a[11], &window) || !as_int(a[12], &sinks) ||
      !shape_of(a[0], 3, qs) || !shape_of(a[5], 2, ts) || !shape_of(a[10], 1, &ws))
    return other_path();
  at = k.at;
  if (k.layered || v.layered || v.at != at || v.dim != k.dim || v.slots != k.slots ||
      qs[2] != 128 || qs[1] > INT_MAX)
    return other_path();
  const double scale = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return other_path();
  const int64_t table_shape[2] = {qs[0], ts[1]};
  if (!has_dtype(a[0], t_bf16) || !placed(a[0], at, &q) ||
      (a[3] != Py_None && !want(a[3], t_i8, 1, &k.dim, at, &ksg)) ||
      (a[4] != Py_None && !want(a[4], t_i8, 1, &k.dim, at, &vsg)) ||
      !want(a[5], t_i32, 2, table_shape, at, &table) || !want(a[7], t_i32, 1, qs, at, &lens) ||
      !want(a[9], t_bf16, 3, qs, at, &out) || !has_dtype(a[10], t_u8) ||
      !placed(a[10], at, &work) || !stream_of(a[13], at, &stream))
    return other_path();
  kq_status st;
  Py_BEGIN_ALLOW_THREADS
  st = c_attn(q, qs[0], (int)qs[1], (int)(k.dim / 128), ksg, vsg, k.p[0], k.p[1], k.p[2], v.p[0],
              v.p[1], v.p[2], k.slots, table, ts[1], page, lens, window, sinks, (float)scale, out,
              work, (size_t)ws, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// copy(pairs, page_size, k_cache, v_cache or None, stream)
static PyObject* copy(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  Cache k, v = {{NULL, NULL, NULL}, 0, 0, 0, 0, 0};
  int page;
  int64_t ps[2];
  void *pairs, *stream;
  if (n_args != 5 || !c_copy || !cache_of(a[2], &k) || !as_int(a[1], &page) ||
      !shape_of(a[0], 2, ps) || ps[1] != 2)
    return other_path();
  if (a[3] != Py_None && (!cache_of(a[3], &v) || v.dim != k.dim || v.slots != k.slots ||
                          v.layers != k.layers || v.at != k.at))
    return other_path();
  if (!has_dtype(a[0], t_i32) || !placed(a[0], k.at, &pairs) || !stream_of(a[4], k.at, &stream))
    return other_path();
  kq_status st;
  Py_BEGIN_ALLOW_THREADS
  st = c_copy(pairs, ps[0], page, k.slots, (int)k.layers, (int)k.dim, k.p[0], k.p[1], k.p[2],
              v.p[0], v.p[1], v.p[2], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// init(bf16, f32, f16, u8, i8, i32, current raw stream, current device, and the
// addresses of kq_gemv, kq_attn_decode_int4_kv and kq_kv_copy_pages)
static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  PyObject** to[8] = {&t_bf16, &t_f32, &t_f16, &t_u8, &t_i8, &t_i32, &f_stream, &f_device};
  void* fn[3];
  if (n_args != 11) {
    PyErr_SetString(PyExc_TypeError, "init takes 11 arguments");
    return NULL;
  }
  for (int i = 0; i < 3; ++i) {
    fn[i] = PyLong_AsVoidPtr(a[8 + i]);
    if (PyErr_Occurred()) return NULL;
  }
  for (int i = 0; i < 8; ++i) Py_XSETREF(*to[i], Py_NewRef(a[i]));
  c_gemv = (__typeof__(&kq_gemv))fn[0];
  c_attn = (__typeof__(&kq_attn_decode_int4_kv))fn[1];
  c_copy = (__typeof__(&kq_kv_copy_pages))fn[2];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, NULL},
    {"gemv", (PyCFunction)(void (*)(void))gemv, METH_FASTCALL, NULL},
    {"attn", (PyCFunction)(void (*)(void))attn, METH_FASTCALL, NULL},
    {"copy", (PyCFunction)(void (*)(void))copy, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {
    PyModuleDef_HEAD_INIT, "_kq_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__kq_call(void) {
  PyObject** names[] = {&n_dtype, &n_shape, &n_get_device, &n_is_contiguous,
                        &n_data_ptr, &n_cuda_stream, &n_view};
  const char* text[] = {"dtype", "shape", "get_device", "is_contiguous",
                        "data_ptr", "cuda_stream", "_view"};
  for (int i = 0; i < 7; ++i)
    if (!(*names[i] = PyUnicode_InternFromString(text[i]))) return NULL;
  return PyModule_Create(&module);
}
