// calls.cpp -- argument marshalling of the ragged-chunk calls as a CPython extension
// module over torch's tensors: device pointers and the current stream taken from
// them, the C entry point called, its status returned.  These calls are made for every
// chunk and layer on kernels of a few microseconds: through ctypes a plan spent 6.9 us
// on the host for 4.8 us on the device.
//
// Their lengths come from the caller's tensors, so every tensor is checked for what the
// call reads or writes there: type, contiguous values, as many of them as the geometry
// and the counts ask for, one device for all and that the current one.  Reading that from
// the tensors themselves costs a few nanoseconds each; from Python methods it would be a
// plan's 15 tensors times four calls.
//
// bind() receives the addresses of the entry points from the loaded library.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <cstring>

#include "../../include/dflash.h"

namespace {

decltype(&dflash_chunk_plan) plan_fn;
decltype(&dflash_chunk_rope_store) rope_fn;
decltype(&dflash_chunk_attention) attn_fn;
PyObject *s_cuda_stream, *out_keys[9];
const char *const kOutKeys[9] = {"cu_rows", "n_pages", "alloc_limit", "seq_lens", "free_head",
                                 "row_req", "row_pos", "row_page",    "row_slot"};

struct PythonError {};  // thrown with Python's error set

template <class... A>
[[noreturn]] void refuse(PyObject *type, const char *format, A... a) {
  PyErr_Format(type, format, a...);
  throw PythonError{};
}

// The memory of a ctypes structure.
template <class T>
struct Structure {
  Py_buffer b{};
  explicit Structure(PyObject *o) {
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) < 0) throw PythonError{};
    if (static_cast<size_t>(b.len) < sizeof(T)) {
      PyBuffer_Release(&b);
      refuse(PyExc_TypeError, "structure of another type");
    }
  }
  Structure(const Structure &) = delete;
  ~Structure() { PyBuffer_Release(&b); }
  const T *get() const { return static_cast<const T *>(b.buf); }
};

int integer(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v < INT32_MIN || v > INT32_MAX)
    refuse(PyExc_OverflowError, "argument does not fit 32 bits");
  return static_cast<int>(v);
}

// The values that n things of each size take, in floating point: a geometry that makes
// no sense (refused by the entry point) must not overflow.
double product(double a, double b, double c = 1, double d = 1, double e = 1) {
  return a * b * c * d * e;
}

// A call's tensors, checked as their addresses are taken.  None gives null, which the
// entry points refuse where they need the buffer.
class Tensors {
 public:
  // A tensor of `need` contiguous values at least.
  template <class T = void>
  T *dense(PyObject *o, const char *name, at::ScalarType type, double need) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = checked(o, name, type);
    if (!t.is_contiguous()) refuse(PyExc_AssertionError, "%s: tensor is not contiguous", name);
    if (static_cast<double>(t.numel()) < need)
      refuse(PyExc_ValueError, "%s: tensor is shorter than the call's counts ask for", name);
    return static_cast<T *>(t.mutable_data_ptr());
  }
  int32_t *ints(PyObject *o, const char *name, double need) {
    return dense<int32_t>(o, name, at::kInt, need);
  }
  // Rows of `width` bf16 values at least, n of them: any step between rows, the rest of a
  // row contiguous ([rows, values] or [rows, heads, dims]).
  void *rows(PyObject *o, const char *name, int64_t n, int64_t width, int64_t *step) {
    *step = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor &t = checked(o, name, at::kBFloat16);
    const int64_t d = t.dim();
    if (d < 2 || d > 3 || (t.stride(d - 1) != 1 && t.size(d - 1) > 1) ||
        (d == 3 && t.stride(1) != t.size(2) && t.size(1) > 1))
      refuse(PyExc_AssertionError, "%s: rows are not contiguous", name);
    if (t.size(0) < n)
      refuse(PyExc_ValueError, "%s: tensor has fewer rows than the call", name);
    if (t.size(1) * (d == 3 ? t.size(2) : 1) < width)
      refuse(PyExc_ValueError, "%s: rows are shorter than the geometry's heads", name);
    *step = t.stride(0);
    return t.mutable_data_ptr();
  }
  // Scratch memory of any type.
  void *scratch(PyObject *o, const char *name, size_t *bytes) {
    *bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor &t = checked(o, name, at::ScalarType::Undefined);
    if (!t.is_contiguous()) refuse(PyExc_AssertionError, "%s: tensor is not contiguous", name);
    *bytes = t.nbytes();
    return t.mutable_data_ptr();
  }
  // The stream asked for, or the current one, of the tensors' device.
  dflash_stream_t stream(PyObject *s) const {
    if (mixed_) refuse(PyExc_ValueError, "tensors are on different devices");
    if (!device_.is_cuda() || device_.index() != c10::cuda::current_device())
      refuse(PyExc_ValueError, "tensors are not on the current CUDA device");
    if (s == Py_None) return c10::cuda::getCurrentCUDAStream(device_.index()).stream();
    PyObject *o = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttr(s, s_cuda_stream);
    if (!o) throw PythonError{};
    void *p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    if (!p && PyErr_Occurred()) throw PythonError{};
    return static_cast<dflash_stream_t>(p);
  }

 private:
  const at::Tensor &checked(PyObject *o, const char *name, at::ScalarType type) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s: not a tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (type != at::ScalarType::Undefined && t.scalar_type() != type)
      refuse(PyExc_TypeError, "%s: tensor of %s expected, of %s given", name, at::toString(type),
             at::toString(t.scalar_type()));
    if (!any_) device_ = t.device();
    mixed_ |= t.device() != device_;
    any_ = true;
    return t;
  }
  c10::Device device_{c10::kCPU};
  bool any_ = false, mixed_ = false;
};

// A tensor's first dimension, as one of the call's counts.
int count(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s: not a tensor", name);
  const at::Tensor &t = THPVariable_Unpack(o);
  const int64_t n = t.dim() > 0 ? t.size(0) : 0;
  if (n > INT32_MAX) refuse(PyExc_ValueError, "%s: dimension does not fit a 32-bit count", name);
  return static_cast<int>(n);
}

// The plan's outputs, from a mapping.
struct Fields {
  PyObject *o[9] = {};
  explicit Fields(PyObject *mapping) {
    for (int i = 0; i < 9; ++i)
      if (!(o[i] = PyObject_GetItem(mapping, out_keys[i]))) {
        while (i > 0) Py_DECREF(o[--i]);
        throw PythonError{};
      }
  }
  Fields(const Fields &) = delete;
  ~Fields() {
    for (PyObject *x : o) Py_DECREF(x);
  }
};

// A KV pool's values, or none where the geometry has another kind (refused).
double pool_values(const dflash_geom *g) {
  if (g->kind != DFLASH_KIND_GQA) return 0;
  return 2.0 * product(g->num_layers, g->num_pool_pages, g->nkv, g->page_size, g->head_dim);
}
int64_t row_width(const dflash_geom *g, int heads) {
  return g->kind == DFLASH_KIND_GQA ? static_cast<int64_t>(heads) * g->head_dim : 0;
}

// The entry point called without the interpreter's lock: a launch waits where the GPU's
// queue is full, and what it waits for may need another Python thread.
template <class F>
PyObject *unlocked(F f) {
  PyThreadState *saved = PyEval_SaveThread();
  const int rc = f();  // a C entry point: no exceptions
  PyEval_RestoreThread(saved);
  return PyLong_FromLong(rc);
}

// A call with `want` arguments; C++ exceptions become Python's.
template <class F>
PyObject *call(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) refuse(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
    return f();
  } catch (const PythonError &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// geom, n_new, ctx_len, n_pages, block_table, free_pages, free_range, valid, max_ctx, out,
// dev_status, stream
PyObject *chunk_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 12, [&] {
    const Structure<dflash_geom> geom(a[0]);
    const dflash_geom *g = geom.get();
    Tensors t;
    const int B = count(a[1], "n_new"), n_free = count(a[5], "free_pages");
    const int32_t *n_new = t.ints(a[1], "n_new", B), *ctx = t.ints(a[2], "ctx_len", B),
                  *have = t.ints(a[3], "n_pages", B);
    int32_t *tbl = t.ints(a[4], "block_table", product(B, g->max_pages));
    const int32_t *free_pages = t.ints(a[5], "free_pages", n_free),
                  *range = t.ints(a[6], "free_range", 2);
    const bool flags = a[7] != Py_None && THPVariable_Check(a[7]) &&
                       THPVariable_Unpack(a[7]).scalar_type() == at::kBool;
    const uint8_t *valid = t.dense<uint8_t>(a[7], "valid", flags ? at::kBool : at::kByte, B);
    const int max_ctx = integer(a[8]);
    int32_t *st = t.ints(a[10], "dev_status", 1), *o[9];
    const Fields fields(a[9]);
    const int n_rows = count(fields.o[5], kOutKeys[5]);
    for (int i = 0; i < 9; ++i)
      o[i] = t.ints(fields.o[i], kOutKeys[i], i == 0 ? B + 1.0 : i < 4 ? B : i == 4 ? 1 : n_rows);
    const dflash_stream_t stream = t.stream(a[11]);
    const dflash_chunk_outputs out = {o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7], o[8]};
    return unlocked([&] {
      return plan_fn(g, B, n_rows, n_new, ctx, have, tbl, free_pages, n_free, range, valid, max_ctx,
                     &out, st, stream);
    });
  });
}

// geom, layer, rope, q, k, v, row_pos, row_page, row_slot, q_out, kv_pool, gamma_q, gamma_k,
// dev_status, stream
PyObject *chunk_rope_store(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 15, [&] {
    const Structure<dflash_geom> geom(a[0]);
    const Structure<dflash_rope_spec> spec(a[2]);
    const dflash_geom *g = geom.get();
    const int layer = integer(a[1]), n_rows = count(a[6], "row_pos");
    const int64_t wq = row_width(g, g->hq), wk = row_width(g, g->nkv);
    int64_t qs, ks, vs, os;
    Tensors t;
    const void *q = t.rows(a[3], "q", n_rows, wq, &qs), *k = t.rows(a[4], "k", n_rows, wk, &ks),
               *v = t.rows(a[5], "v", n_rows, wk, &vs);
    const int32_t *pos = t.ints(a[6], "row_pos", n_rows), *page = t.ints(a[7], "row_page", n_rows),
                  *slot = t.ints(a[8], "row_slot", n_rows);
    void *q_out = t.rows(a[9], "q_out", n_rows, wq, &os);
    void *pool = t.dense(a[10], "kv_pool", at::kBFloat16, pool_values(g));
    const void *gq = t.dense(a[11], "gamma_q", at::kBFloat16, g->head_dim),
               *gk = t.dense(a[12], "gamma_k", at::kBFloat16, g->head_dim);
    int32_t *st = t.ints(a[13], "dev_status", 1);
    const dflash_stream_t stream = t.stream(a[14]);
    return unlocked([&] {
      return rope_fn(g, layer, n_rows, spec.get(), q, qs, k, ks, v, vs, gq, gk, pos, page, slot,
                     q_out, os, pool, st, stream);
    });
  });
}

// geom, layer, q, kv_pool, block_table, cu_rows, ctx_len, kv_len, out, workspace, window, sinks,
// scale, mask_mode, num_segments, dev_status, stream
PyObject *chunk_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 17, [&] {
    const Structure<dflash_geom> geom(a[0]);
    const dflash_geom *g = geom.get();
    const int layer = integer(a[1]), n_rows = count(a[2], "q"), B = count(a[7], "kv_len");
    const int64_t wq = row_width(g, g->hq);
    int64_t qs, os;
    size_t ws_bytes;
    Tensors t;
    const void *q = t.rows(a[2], "q", n_rows, wq, &qs);
    const void *pool = t.dense(a[3], "kv_pool", at::kBFloat16, pool_values(g));
    const int32_t *tbl = t.ints(a[4], "block_table", product(B, g->max_pages)),
                  *cu = t.ints(a[5], "cu_rows", B + 1.0), *ctx = t.ints(a[6], "ctx_len", B),
                  *kv = t.ints(a[7], "kv_len", B);
    void *out = t.rows(a[8], "out", n_rows, wq, &os);
    void *ws = t.scratch(a[9], "workspace", &ws_bytes);
    const int window = integer(a[10]);
    const float *sinks = t.dense<float>(a[11], "sinks", at::kFloat, g->hq);
    const double scale = a[12] == Py_None ? 0.0 : PyFloat_AsDouble(a[12]);
    if (scale == -1.0 && PyErr_Occurred()) throw PythonError{};
    const int mode = integer(a[13]), segments = integer(a[14]);
    int32_t *st = t.ints(a[15], "dev_status", 1);
    const dflash_stream_t stream = t.stream(a[16]);
    return unlocked([&] {
      return attn_fn(g, B, layer, n_rows, q, qs, pool, tbl, cu, ctx, kv, window, sinks,
                     static_cast<float>(scale), mode, segments, ws, ws_bytes, out, os, st, stream);
    });
  });
}

// plan, rope and attention addresses
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 3, [&] {
    void *f[3];
    for (int i = 0; i < 3; ++i) {
      f[i] = PyLong_AsVoidPtr(a[i]);
      if (!f[i] && PyErr_Occurred()) throw PythonError{};
      if (!f[i]) refuse(PyExc_ValueError, "null entry point");
    }
    std::memcpy(&plan_fn, &f[0], sizeof f[0]);
    std::memcpy(&rope_fn, &f[1], sizeof f[1]);
    std::memcpy(&attn_fn, &f[2], sizeof f[2]);
    return Py_NewRef(Py_None);
  });
}

using Method = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);
PyCFunction method(Method m) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(m));
}
PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"chunk_plan", method(chunk_plan), METH_FASTCALL, nullptr},
    {"chunk_rope_store", method(chunk_rope_store), METH_FASTCALL, nullptr},
    {"chunk_attention", method(chunk_attention), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__calls(void) {
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!s_cuda_stream) return nullptr;
  for (int i = 0; i < 9; ++i)
    if (!(out_keys[i] = PyUnicode_InternFromString(kOutKeys[i]))) return nullptr;
  PyObject *m = PyModule_Create(&module);
  // tensors are read as the torch it was compiled against lays them out
  if (m && PyModule_AddStringConstant(m, "torch_version", DFLASH_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
