/* fastcall.c -- the 4-bit, block-norm and attention entry points called from Python without ctypes.
 *
 * A product of one token takes some 6 us on the GPU. A call of it through ctypes and its Python wrapper takes 4.9 us of
 * the host's time, 2.3 of them inside the library (Grace); through this module 3.1. Same functions, names, argument
 * order, defaults and refusals as the ctypes wrappers of __init__.py, which stay and are used where this module could not
 * be built; an argument of a wrong type is a TypeError here and a ctypes.ArgumentError there. The library's functions come
 * in as addresses (init), so nothing is linked. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "fp8gb.h"

enum { QUANTIZE, DEQUANTIZE, SCALED_MM, NORM_FWD, NORM_BWD, ROPE_FWD, ROPE_BWD, APPEND, ATTENTION, COUNT };
static void* g_fn[COUNT];
static PyObject *g_error, *g_stream, *g_raw, *g_device; /* callables: of a status; of None; of a device; of nothing */
static PyObject *g_state, *g_norm, *g_grad, *g_rope, *g_rope_grad, *g_cache, *g_batch, *g_attention; /* the classes of the ctypes structures */
static PyObject *s_data_ptr, *s_cuda_stream, *s_c;

/* Arguments by position, then by name, into out[n]; what is left out stays NULL and must not be required. */
static int take(const char* who, const char* const* names, int n, int required, PyObject* const* args, Py_ssize_t nargs, PyObject* kw, PyObject** out) {
  if (nargs > n) {
    PyErr_Format(PyExc_TypeError, "%s takes at most %d arguments (%zd given)", who, n, nargs);
    return 0;
  }
  for (int i = 0; i < n; ++i) out[i] = i < nargs ? args[i] : NULL;
  const Py_ssize_t nkw = kw != NULL ? PyTuple_GET_SIZE(kw) : 0;
  for (Py_ssize_t k = 0; k < nkw; ++k) {
    int i = 0;
    while (i < n && PyUnicode_CompareWithASCIIString(PyTuple_GET_ITEM(kw, k), names[i]) != 0) ++i;
    if (i == n || out[i] != NULL) {
      PyErr_Format(PyExc_TypeError, "%s got %s argument '%U'", who, i == n ? "an unexpected" : "twice the", PyTuple_GET_ITEM(kw, k));
      return 0;
    }
    out[i] = args[nargs + k];
  }
  for (int i = 0; i < required; ++i)
    if (out[i] == NULL) {
      PyErr_Format(PyExc_TypeError, "%s misses its argument '%s'", who, names[i]);
      return 0;
    }
  return 1;
}

/* None, an address, or a tensor. */
static int pointer(PyObject* o, void** p) {
  *p = NULL;
  if (o == NULL || o == Py_None) return 1;
  if (PyLong_Check(o)) {
    *p = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
  }
  PyObject* r = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (r == NULL) return 0;
  *p = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

/* The address of an instance of a ctypes structure. Nothing else is taken: the library reads the whole of it. */
static int structure(PyObject* o, PyObject* type, void** p) {
  *p = NULL;
  if (o == NULL || o == Py_None) return 1;
  const int is = PyObject_IsInstance(o, type);
  if (is < 0) return 0;
  if (!is) {
    PyErr_Format(PyExc_TypeError, "expected %s, not %s", ((PyTypeObject*)type)->tp_name, Py_TYPE(o)->tp_name);
    return 0;
  }
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) return 0;
  *p = b.buf;
  PyBuffer_Release(&b);
  return 1;
}

/* A tensor's state, or an object that has one in its attribute c; *keep holds it over the call. */
static int state(PyObject* o, void** p, PyObject** keep) {
  *keep = NULL;
  if (o != NULL && o != Py_None && !Py_IS_TYPE(o, (PyTypeObject*)g_state)) {
    const int is = PyObject_IsInstance(o, g_state);
    if (is < 0) return 0;
    if (!is && (o = *keep = PyObject_GetAttr(o, s_c)) == NULL) return 0;
  }
  if (structure(o, g_state, p)) return 1;
  Py_CLEAR(*keep);
  return 0;
}

static int integer(PyObject* o, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  return *v != -1 || !PyErr_Occurred();
}

static int integer32(PyObject* o, int* v) {
  int64_t w;
  if (!integer(o, &w)) return 0;
  if (w < INT32_MIN || w > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
    return 0;
  }
  *v = (int)w;
  return 1;
}

/* A stream: None (torch's current one), a raw handle, or an object with one. */
static int stream(PyObject* o, void** p) {
  PyObject* r;
  if (o == NULL || o == Py_None) {
    if (g_raw != NULL) {
      PyObject* d = PyObject_CallNoArgs(g_device);
      if (d == NULL) return 0;
      r = PyObject_CallOneArg(g_raw, d);
      Py_DECREF(d);
    } else {
      r = PyObject_CallOneArg(g_stream, Py_None);
    }
  } else {
    r = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttr(o, s_cuda_stream);
  }
  if (r == NULL) return 0;
  *p = r == Py_None ? NULL : PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

/* 0 as the wrappers return it, or the exception that the status stands for. */
static PyObject* status(fp8_status_t s) {
  if (s == FP8_OK) return PyLong_FromLong(0);
  return PyObject_CallFunction(g_error, "i", (int)s);
}

#define CALL(s, call)    \
  do {                   \
    Py_BEGIN_ALLOW_THREADS s = call; \
    Py_END_ALLOW_THREADS \
  } while (0)

static PyObject* quantize(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"x", "rows", "cols", "ld", "fmt", "mode", "st", "q", "sf", "qT", "sfT", "stream"};
  PyObject* a[12];
  void *x, *st, *q, *sf, *qT, *sfT, *s;
  int64_t rows, cols, ld;
  int fmt, mode;
  PyObject* keep;
  (void)self;
  if (!take("fp4_quantize", names, 12, 9, args, nargs, kw, a) || !pointer(a[0], &x) || !integer(a[1], &rows) || !integer(a[2], &cols) ||
      !integer(a[3], &ld) || !integer32(a[4], &fmt) || !integer32(a[5], &mode) || !pointer(a[7], &q) || !pointer(a[8], &sf) || !pointer(a[9], &qT) ||
      !pointer(a[10], &sfT) || !stream(a[11], &s) || !state(a[6], &st, &keep))
    return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const void*, int64_t, int64_t, int64_t, fp4_format_t, fp8_scaling_t, const fp8_tensor_state_t*, void*, void*, void*, void*,
                            void*))g_fn[QUANTIZE])(x, rows, cols, ld, (fp4_format_t)fmt, (fp8_scaling_t)mode, st, q, sf, qT, sfT, s));
  Py_XDECREF(keep);
  return status(r);
}

static PyObject* dequantize(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"q", "sf", "MN", "K", "fmt", "scale_inv", "y", "dt", "ldy", "stream"};
  PyObject* a[10];
  void *q, *sf, *d, *y, *s;
  int64_t mn, k, ldy;
  int fmt, dt;
  (void)self;
  if (!take("fp4_dequantize", names, 10, 9, args, nargs, kw, a) || !pointer(a[0], &q) || !pointer(a[1], &sf) || !integer(a[2], &mn) || !integer(a[3], &k) ||
      !integer32(a[4], &fmt) || !pointer(a[5], &d) || !pointer(a[6], &y) || !integer32(a[7], &dt) || !integer(a[8], &ldy) || !stream(a[9], &s))
    return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const void*, const void*, int64_t, int64_t, fp4_format_t, const float*, void*, fp8_dtype_t, int64_t, void*))g_fn[DEQUANTIZE])(
              q, sf, mn, k, (fp4_format_t)fmt, d, y, (fp8_dtype_t)dt, ldy, s));
  return status(r);
}

static PyObject* scaled_mm(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"A", "sfa", "B", "sfb", "M", "N", "K", "fmt", "scale_inv_a", "scale_inv_b", "C", "dt", "ldc", "stream"};
  PyObject* a[14];
  void *A, *sfa, *B, *sfb, *da, *db, *C, *s;
  int64_t m, n, k, ldc;
  int fmt, dt;
  (void)self;
  if (!take("fp4_scaled_mm", names, 14, 13, args, nargs, kw, a) || !pointer(a[0], &A) || !pointer(a[1], &sfa) || !pointer(a[2], &B) || !pointer(a[3], &sfb) ||
      !integer(a[4], &m) || !integer(a[5], &n) || !integer(a[6], &k) || !integer32(a[7], &fmt) || !pointer(a[8], &da) || !pointer(a[9], &db) ||
      !pointer(a[10], &C) || !integer32(a[11], &dt) || !integer(a[12], &ldc) || !stream(a[13], &s))
    return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const void*, const void*, const void*, const void*, int64_t, int64_t, int64_t, fp4_format_t, const float*, const float*, void*,
                            fp8_dtype_t, int64_t, void*))g_fn[SCALED_MM])(A, sfa, B, sfb, m, n, k, (fp4_format_t)fmt, da, db, C, (fp8_dtype_t)dt, ldc, s));
  return status(r);
}

static PyObject* norm_fwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"f", "stream"};
  PyObject* a[2];
  void *f, *s;
  (void)self;
  if (!take("fp8_block_norm_fwd", names, 2, 1, args, nargs, kw, a) || !structure(a[0], g_norm, &f) || !stream(a[1], &s)) return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const fp8_block_norm_t*, void*))g_fn[NORM_FWD])(f, s));
  return status(r);
}

static PyObject* norm_bwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"f", "b", "workspace", "workspace_bytes", "stream"};
  PyObject* a[5];
  void *f, *b, *w, *s;
  int64_t n;
  (void)self;
  if (!take("fp8_block_norm_bwd", names, 5, 4, args, nargs, kw, a) || !structure(a[0], g_norm, &f) || !structure(a[1], g_grad, &b) || !pointer(a[2], &w) ||
      !integer(a[3], &n) || !stream(a[4], &s))
    return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const fp8_block_norm_t*, const fp8_block_norm_grad_t*, void*, int64_t, void*))g_fn[NORM_BWD])(f, b, w, n, s));
  return status(r);
}

static PyObject* rope_fwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"f", "stream"};
  PyObject* a[2];
  void *f, *s;
  (void)self;
  if (!take("fp8_qk_rope_fwd", names, 2, 1, args, nargs, kw, a) || !structure(a[0], g_rope, &f) || !stream(a[1], &s)) return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const fp8_qk_rope_t*, void*))g_fn[ROPE_FWD])(f, s));
  return status(r);
}

static PyObject* rope_bwd(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"f", "b", "workspace", "workspace_bytes", "stream"};
  PyObject* a[5];
  void *f, *b, *w, *s;
  int64_t n;
  (void)self;
  if (!take("fp8_qk_rope_bwd", names, 5, 4, args, nargs, kw, a) || !structure(a[0], g_rope, &f) || !structure(a[1], g_rope_grad, &b) || !pointer(a[2], &w) ||
      !integer(a[3], &n) || !stream(a[4], &s))
    return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const fp8_qk_rope_t*, const fp8_qk_rope_grad_t*, void*, int64_t, void*))g_fn[ROPE_BWD])(f, b, w, n, s));
  return status(r);
}

static PyObject* append(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"f", "cache", "batch", "stream"};
  PyObject* a[4];
  void *f, *c, *b, *s;
  (void)self;
  if (!take("fp8_kv_append", names, 4, 3, args, nargs, kw, a) || !structure(a[0], g_rope, &f) || !structure(a[1], g_cache, &c) || !structure(a[2], g_batch, &b) ||
      !stream(a[3], &s))
    return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const fp8_qk_rope_t*, const fp8_kv_cache_t*, const fp8_kv_batch_t*, void*))g_fn[APPEND])(f, c, b, s));
  return status(r);
}

static PyObject* attention(PyObject* self, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  static const char* const names[] = {"a", "cache", "batch", "workspace", "workspace_bytes", "stream"};
  PyObject* a[6];
  void *f, *c, *b, *w, *s;
  int64_t n;
  (void)self;
  if (!take("fp8_paged_attention", names, 6, 5, args, nargs, kw, a) || !structure(a[0], g_attention, &f) || !structure(a[1], g_cache, &c) ||
      !structure(a[2], g_batch, &b) || !pointer(a[3], &w) || !integer(a[4], &n) || !stream(a[5], &s))
    return NULL;
  fp8_status_t r;
  CALL(r, ((fp8_status_t(*)(const fp8_paged_attention_t*, const fp8_kv_cache_t*, const fp8_kv_batch_t*, void*, int64_t, void*))g_fn[ATTENTION])(f, c, b, w, n, s));
  return status(r);
}

/* init((addresses in the order above), error callable, stream callable, (classes of the state, the norm, its gradients, the heads, their
 * gradients, the cache, the batch, the attention)) */
static PyObject* init(PyObject* self, PyObject* args) {
  PyObject *addresses, *error, *current;
  PyTypeObject* classes[8];
  PyObject** const held[8] = {&g_state, &g_norm, &g_grad, &g_rope, &g_rope_grad, &g_cache, &g_batch, &g_attention};
  (void)self;
  if (!PyArg_ParseTuple(args, "O!OO(O!O!O!O!O!O!O!O!)", &PyTuple_Type, &addresses, &error, &current, &PyType_Type, &classes[0], &PyType_Type, &classes[1],
                        &PyType_Type, &classes[2], &PyType_Type, &classes[3], &PyType_Type, &classes[4], &PyType_Type, &classes[5], &PyType_Type, &classes[6],
                        &PyType_Type, &classes[7]))
    return NULL;
  if (PyTuple_GET_SIZE(addresses) != COUNT) {
    PyErr_SetString(PyExc_ValueError, "one address per function");
    return NULL;
  }
  for (int i = 0; i < COUNT; ++i) {
    g_fn[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
    if (PyErr_Occurred()) return NULL;
  }
  Py_XSETREF(g_error, Py_NewRef(error));
  Py_XSETREF(g_stream, Py_NewRef(current));
  for (int i = 0; i < 8; ++i) Py_XSETREF(*held[i], Py_NewRef((PyObject*)classes[i]));
  Py_RETURN_NONE;
}

/* use_torch(raw stream of a device, current device): where there is a GPU */
static PyObject* use_torch(PyObject* self, PyObject* args) {
  PyObject *raw, *device;
  (void)self;
  if (!PyArg_ParseTuple(args, "OO", &raw, &device)) return NULL;
  Py_XSETREF(g_raw, Py_NewRef(raw));
  Py_XSETREF(g_device, Py_NewRef(device));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, NULL},
    {"use_torch", use_torch, METH_VARARGS, NULL},
    {"fp4_quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL | METH_KEYWORDS, NULL},
    {"fp4_dequantize", (PyCFunction)(void (*)(void))dequantize, METH_FASTCALL | METH_KEYWORDS, NULL},
    {"fp4_scaled_mm", (PyCFunction)(void (*)(void))scaled_mm, METH_FASTCALL | METH_KEYWORDS, NULL},
    {"fp8_block_norm_fwd", (PyCFunction)(void (*)(void))norm_fwd, METH_FASTCALL | METH_KEYWORDS, NULL},
    {"fp8_block_norm_bwd", (PyCFunction)(void (*)(void))norm_bwd, METH_FASTCALL | METH_KEYWORDS, NULL},
    {"fp8_qk_rope_fwd", (PyCFunction)(void (*)(void))rope_fwd, METH_FASTCALL | METH_KEYWORDS, NULL},
    {"fp8_qk_rope_bwd", (PyCFunction)(void (*)(void))rope_bwd, METH_FASTCALL | METH_KEYWORDS, NULL},
    {"fp8_kv_append", (PyCFunction)(void (*)(void))append, METH_FASTCALL | METH_KEYWORDS, NULL},
    {"fp8_paged_attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL | METH_KEYWORDS, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  s_c = PyUnicode_InternFromString("c");
  return s_data_ptr && s_cuda_stream && s_c ? PyModule_Create(&module) : NULL;
}
