/* calls.c -- argument marshalling of the ragged-chunk calls as a CPython
 * extension module: the same as the ctypes bindings' (tensors to device pointers,
 * the current torch stream to a cudaStream_t, the C entry point called, its status
 * returned), at a fraction of their cost.  These calls are made for every chunk
 * and layer on kernels of a few microseconds: through ctypes a plan spent 6.9 us
 * on the host for 4.8 us on the device.
 *
 * bind() receives the addresses of the entry points from the loaded library, and
 * torch's two functions for the current device and stream.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../include/dflash.h"

static int (*plan_fn)(const dflash_geom *, int, int, const int32_t *, const int32_t *,
                      const int32_t *, int32_t *, const int32_t *, int, const int32_t *,
                      const uint8_t *, int32_t, const dflash_chunk_outputs *, int32_t *,
                      dflash_stream_t);
static int (*rope_fn)(const dflash_geom *, int, int, const dflash_rope_spec *, const void *, int64_t,
                      const void *, int64_t, const void *, int64_t, const void *, const void *,
                      const int32_t *, const int32_t *, const int32_t *, void *, int64_t, void *,
                      int32_t *, dflash_stream_t);
static int (*attn_fn)(const dflash_geom *, int, int, int, const void *, int64_t, const void *,
                      const int32_t *, const int32_t *, const int32_t *, const int32_t *, int32_t,
                      const float *, float, int, int, void *, size_t, void *, int64_t, int32_t *,
                      dflash_stream_t);
static PyObject *current_device, *current_stream;
static PyObject *s_data_ptr, *s_size, *s_stride, *s_is_contiguous, *s_get_device, *s_cuda_stream,
    *s_nbytes, *zero;
static PyObject *out_keys[9];
static const char *const kOutKeys[9] = {"cu_rows", "n_pages", "alloc_limit",
                                        "seq_lens", "free_head", "row_req",
                                        "row_pos", "row_page", "row_slot"};

/* Address of a tensor's data; None gives NULL. */
static int addr(PyObject *t, void *out) {
  void **p = (void **)out;
  if (t == Py_None) {
    *p = NULL;
    return 0;
  }
  PyObject *o = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!o) return -1;
  *p = PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return *p == NULL && PyErr_Occurred() ? -1 : 0;
}

/* A tensor's first dimension. */
static int length(PyObject *t, int *out) {
  PyObject *o = PyObject_CallMethodOneArg(t, s_size, zero);
  if (!o) return -1;
  const long long v = PyLong_AsLongLong(o);
  Py_DECREF(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v < 0 || v > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "dimension does not fit a 32-bit count");
    return -1;
  }
  *out = (int)v;
  return 0;
}

static int contiguous(PyObject *t) {
  if (t == Py_None) return 0;
  PyObject *o = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!o) return -1;
  const int yes = PyObject_IsTrue(o);
  Py_DECREF(o);
  if (yes == 0) PyErr_SetString(PyExc_AssertionError, "tensor is not contiguous");
  return yes == 1 ? 0 : -1;
}

/* A row-strided view: its address and the elements between two rows.  Any step
 * between rows, the rest of a row contiguous. */
static int rows(PyObject *t, void *ptr, int64_t *step) {
  *step = 0;
  if (addr(t, ptr) < 0) return -1;
  if (t == Py_None) return 0;
  PyObject *st = PyObject_CallMethodNoArgs(t, s_stride);
  if (!st) return -1;
  int ok = PyTuple_Check(st) && PyTuple_GET_SIZE(st) >= 2;
  const Py_ssize_t n = ok ? PyTuple_GET_SIZE(st) : 0;
  if (ok) {
    *step = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 0));
    ok = PyLong_AsLongLong(PyTuple_GET_ITEM(st, n - 1)) == 1;
  }
  if (ok && n > 2) {
    const long long inner = PyLong_AsLongLong(PyTuple_GET_ITEM(st, 1));
    PyObject *two = PyLong_FromLong(2);
    PyObject *w = two ? PyObject_CallMethodOneArg(t, s_size, two) : NULL;
    Py_XDECREF(two);
    if (!w) {
      Py_DECREF(st);
      return -1;
    }
    ok = PyLong_AsLongLong(w) == inner;
    Py_DECREF(w);
  }
  Py_DECREF(st);
  if (PyErr_Occurred()) return -1;
  if (!ok) PyErr_SetString(PyExc_AssertionError, "rows are not contiguous");
  return ok ? 0 : -1;
}

/* The stream asked for, or the current one of the current device, which has to be
 * the device of `t`. */
static int stream_of(PyObject *s, PyObject *t, dflash_stream_t *out) {
  PyObject *dev = PyObject_CallNoArgs(current_device);
  if (!dev) return -1;
  PyObject *mine = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!mine) {
    Py_DECREF(dev);
    return -1;
  }
  const int same = PyObject_RichCompareBool(dev, mine, Py_EQ);
  Py_DECREF(mine);
  if (same != 1) {
    Py_DECREF(dev);
    if (same == 0) PyErr_SetString(PyExc_ValueError, "tensors are not on the current CUDA device");
    return -1;
  }
  PyObject *o;
  if (s == Py_None) {
    o = PyObject_CallOneArg(current_stream, dev);
  } else if (PyLong_Check(s)) {
    o = Py_NewRef(s);
  } else {
    o = PyObject_GetAttr(s, s_cuda_stream);
  }
  Py_DECREF(dev);
  if (!o) return -1;
  *out = (dflash_stream_t)PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* The memory of a ctypes structure. */
static int structure(PyObject *o, size_t bytes, Py_buffer *b) {
  if (PyObject_GetBuffer(o, b, PyBUF_SIMPLE) < 0) return -1;
  if ((size_t)b->len >= bytes) return 0;
  PyBuffer_Release(b);
  PyErr_SetString(PyExc_TypeError, "structure of another type");
  return -1;
}

static int integer(PyObject *o, int *out) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
    return -1;
  }
  *out = (int)v;
  return 0;
}

static int arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
  return -1;
}

/* geom, n_new, ctx_len, n_pages, block_table, free_pages, free_range, valid, max_ctx, out,
 * dev_status, stream */
static PyObject *chunk_plan(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  const int32_t *n_new, *ctx, *have, *free_pages, *range;
  const uint8_t *valid;
  int32_t *tbl, *st, *o[9];
  int B, n_rows, n_free, max_ctx;
  dflash_stream_t stream;
  Py_buffer g;
  if (arity(n, 12) < 0 || addr(a[1], &n_new) < 0 || addr(a[2], &ctx) < 0 || addr(a[3], &have) < 0 ||
      contiguous(a[4]) < 0 || addr(a[4], &tbl) < 0 || addr(a[5], &free_pages) < 0 ||
      addr(a[6], &range) < 0 || addr(a[7], &valid) < 0 || integer(a[8], &max_ctx) < 0 ||
      addr(a[10], &st) < 0 || length(a[1], &B) < 0 || length(a[5], &n_free) < 0)
    return NULL;
  for (int i = 0; i < 9; ++i) {
    PyObject *t = PyObject_GetItem(a[9], out_keys[i]);
    if (!t) return NULL;
    const int bad = addr(t, &o[i]) < 0 || (i == 5 && length(t, &n_rows) < 0);
    Py_DECREF(t); /* the mapping keeps it */
    if (bad) return NULL;
  }
  if (stream_of(a[11], a[6], &stream) < 0 || structure(a[0], sizeof(dflash_geom), &g) < 0)
    return NULL;
  const dflash_chunk_outputs out = {o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7], o[8]};
  const int rc = plan_fn((const dflash_geom *)g.buf, B, n_rows, n_new, ctx, have, tbl, free_pages,
                         n_free, range, valid, max_ctx, &out, st, stream);
  PyBuffer_Release(&g);
  return PyLong_FromLong(rc);
}

/* geom, layer, rope, q, k, v, row_pos, row_page, row_slot, q_out, kv_pool, gamma_q, gamma_k,
 * dev_status, stream */
static PyObject *chunk_rope_store(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  const void *q, *k, *v, *gq, *gk;
  void *q_out, *pool;
  const int32_t *pos, *page, *slot;
  int32_t *st;
  int64_t qs, ks, vs, os;
  int layer, n_rows;
  dflash_stream_t stream;
  Py_buffer g, spec;
  if (arity(n, 15) < 0 || integer(a[1], &layer) < 0 || rows(a[3], &q, &qs) < 0 ||
      rows(a[4], &k, &ks) < 0 || rows(a[5], &v, &vs) < 0 || addr(a[6], &pos) < 0 ||
      addr(a[7], &page) < 0 || addr(a[8], &slot) < 0 || rows(a[9], &q_out, &os) < 0 ||
      contiguous(a[10]) < 0 || addr(a[10], &pool) < 0 || addr(a[11], &gq) < 0 ||
      addr(a[12], &gk) < 0 || addr(a[13], &st) < 0 || length(a[6], &n_rows) < 0 ||
      stream_of(a[14], a[6], &stream) < 0 || structure(a[0], sizeof(dflash_geom), &g) < 0)
    return NULL;
  if (structure(a[2], sizeof(dflash_rope_spec), &spec) < 0) {
    PyBuffer_Release(&g);
    return NULL;
  }
  const int rc = rope_fn((const dflash_geom *)g.buf, layer, n_rows,
                         (const dflash_rope_spec *)spec.buf, q, qs, k, ks, v, vs, gq, gk, pos, page,
                         slot, q_out, os, pool, st, stream);
  PyBuffer_Release(&spec);
  PyBuffer_Release(&g);
  return PyLong_FromLong(rc);
}

/* geom, layer, q, kv_pool, block_table, cu_rows, ctx_len, kv_len, out, workspace, window, sinks,
 * scale, mask_mode, num_segments, dev_status, stream */
static PyObject *chunk_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  const void *q, *pool;
  void *out, *ws;
  const int32_t *tbl, *cu, *ctx, *kv;
  const float *sinks;
  int32_t *st;
  int64_t qs, os;
  size_t ws_bytes = 0;
  int layer, B, n_rows, window, mode, segments;
  dflash_stream_t stream;
  Py_buffer g;
  if (arity(n, 17) < 0 || integer(a[1], &layer) < 0 || rows(a[2], &q, &qs) < 0 ||
      contiguous(a[3]) < 0 || addr(a[3], &pool) < 0 || contiguous(a[4]) < 0 ||
      addr(a[4], &tbl) < 0 || addr(a[5], &cu) < 0 || addr(a[6], &ctx) < 0 || addr(a[7], &kv) < 0 ||
      rows(a[8], &out, &os) < 0 || addr(a[9], &ws) < 0 || integer(a[10], &window) < 0 ||
      addr(a[11], &sinks) < 0 || integer(a[13], &mode) < 0 || integer(a[14], &segments) < 0 ||
      addr(a[15], &st) < 0 || length(a[7], &B) < 0 || length(a[2], &n_rows) < 0)
    return NULL;
  const double scale = a[12] == Py_None ? 0.0 : PyFloat_AsDouble(a[12]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  if (ws) {
    PyObject *o = PyObject_GetAttr(a[9], s_nbytes);
    if (!o) return NULL;
    ws_bytes = PyLong_AsSize_t(o);
    Py_DECREF(o);
    if (PyErr_Occurred()) return NULL;
  }
  if (stream_of(a[16], a[2], &stream) < 0 || structure(a[0], sizeof(dflash_geom), &g) < 0)
    return NULL;
  const int rc = attn_fn((const dflash_geom *)g.buf, B, layer, n_rows, q, qs, pool, tbl, cu, ctx,
                         kv, window, sinks, (float)scale, mode, segments, ws, ws_bytes, out, os, st,
                         stream);
  PyBuffer_Release(&g);
  return PyLong_FromLong(rc);
}

/* plan, rope and attention addresses, current_device, current_stream */
static PyObject *bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  (void)self;
  if (arity(n, 5) < 0) return NULL;
  void *f[3];
  for (int i = 0; i < 3; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return NULL;
    }
  }
  *(void **)&plan_fn = f[0];
  *(void **)&rope_fn = f[1];
  *(void **)&attn_fn = f[2];
  Py_XSETREF(current_device, Py_NewRef(a[3]));
  Py_XSETREF(current_stream, Py_NewRef(a[4]));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
    {"chunk_plan", (PyCFunction)(void (*)(void))chunk_plan, METH_FASTCALL, NULL},
    {"chunk_rope_store", (PyCFunction)(void (*)(void))chunk_rope_store, METH_FASTCALL, NULL},
    {"chunk_attention", (PyCFunction)(void (*)(void))chunk_attention, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_size = PyUnicode_InternFromString("size");
  s_stride = PyUnicode_InternFromString("stride");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  s_nbytes = PyUnicode_InternFromString("nbytes");
  zero = PyLong_FromLong(0);
  if (!s_data_ptr || !s_size || !s_stride || !s_is_contiguous || !s_get_device || !s_cuda_stream ||
      !s_nbytes || !zero)
    return NULL;
  for (int i = 0; i < 9; ++i)
    if (!(out_keys[i] = PyUnicode_InternFromString(kOutKeys[i]))) return NULL;
  return PyModule_Create(&module);
}
