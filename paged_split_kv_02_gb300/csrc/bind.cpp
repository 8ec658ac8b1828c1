/* Argument marshalling of the calls of paged_step.h and paged_quant.h: tensors to descriptors,
 * the launch's device and stream, then the library's function.  A serving
 * step makes these calls between kernels of a few microseconds each, and the
 * host's part of a call is more than most of the kernels take: filling ctypes
 * structures in Python took 18-20 us of a GB300's host, asking the tensors
 * through their Python methods 6, this 3 (2 of them the launch).  Nothing is
 * computed here. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstring>
#include <exception>
#include <optional>

#include <torch/csrc/autograd/python_variable.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "paged_quant.h"

#define MAX_TENSORS 12

typedef int (*attn_fn)(const pd_tensor *, const pd_tensor *, const pd_tensor *, const pd_tensor *,
                       const pd_tensor *, const pd_tensor *, pd_tensor *, int, int, int, int, int,
                       int, int, float, int, pd_scratch *, void *, const pd_options *);
typedef int (*prefill_fn)(const pd_tensor *, const pd_tensor *, const pd_tensor *,
                          const pd_tensor *, const pd_tensor *, const pd_tensor *,
                          const pd_tensor *, const pd_prefill_plan_info *, pd_tensor *, int, int,
                          int, int, int, int, float, int, pd_scratch *, void *);
typedef int (*tables_fn)(const pd_tensor *, const pd_tensor *, const pd_tensor *,
                         const pd_tensor *, const pd_tensor *, pd_tensor *, pd_tensor *,
                         pd_tensor *, pd_tensor *, pd_tensor *, pd_tensor *, int, int, void *);
typedef int (*rope_fn)(const pd_tensor *, const pd_tensor *, const pd_tensor *, const pd_tensor *,
                       const pd_tensor *, const pd_tensor *, const uint8_t *, pd_tensor *,
                       pd_tensor *, pd_tensor *, int, int, int, int, int, int, int, void *);
typedef int (*quant_attn_fn)(const pd_tensor *, const pd_tensor *, const pd_tensor *,
                             const pd_tensor *, const pd_tensor *, const pd_tensor *,
                             const pd_tensor *, const pd_tensor *, pd_tensor *, int, int, int, int,
                             int, int, int, float, int, pd_scratch *, void *);
typedef int (*quant_read_fn)(const pd_tensor *, const pd_tensor *, const pd_tensor *,
                             const pd_tensor *, const pd_tensor *, const pd_tensor *,
                             const pd_tensor *, pd_tensor *, pd_tensor *, int, int, int, int,
                             void *);
typedef int (*quant_write_fn)(const pd_tensor *, const pd_tensor *, const pd_tensor *,
                              const pd_tensor *, const pd_tensor *, const pd_tensor *,
                              const uint8_t *, pd_tensor *, pd_tensor *, pd_tensor *, pd_tensor *,
                              pd_tensor *, int, int, int, int, int, int, int, void *);
static attn_fn g_attn;
static prefill_fn g_prefill;
static tables_fn g_tables;
static rope_fn g_rope;
static quant_attn_fn g_quant_attn;
static quant_read_fn g_quant_read;
static quant_write_fn g_quant_write;

/* The descriptor of a tensor; its device's index (-1: not CUDA) in *device. */
static bool fill(PyObject *o, pd_tensor *d, int *device) {
  if (!THPVariable_Check(o)) {
    /* (as the ctypes calls answer) */
    PyErr_Format(PyExc_AttributeError, "a tensor or None is wanted, not '%.200s'",
                 Py_TYPE(o)->tp_name);
    return false;
  }
  const at::Tensor &t = THPVariable_Unpack(o);
  memset(d, 0, sizeof *d);
  d->data = t.data_ptr();
  switch (t.scalar_type()) {
    case at::kHalf: d->dtype = PD_F16; break;
    case at::kBFloat16: d->dtype = PD_BF16; break;
    case at::kInt: d->dtype = PD_I32; break;
    case at::kFloat: d->dtype = PD_F32; break;
    case at::kFloat8_e4m3fn: d->dtype = PD_E4M3; break;
    default: d->dtype = 99; /* a type the library does not take */
  }
  const at::IntArrayRef shape = t.sizes(), stride = t.strides();
  d->ndim = (int32_t)shape.size();
  for (size_t i = 0; i < shape.size() && i < 4; ++i) {
    d->shape[i] = shape[i];
    d->stride[i] = stride[i];
  }
  *device = t.device().is_cuda() ? t.device().index() : -1;
  return true;
}

/* The interpreter's lock, let go for a scope. */
struct unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~unlocked() { PyEval_RestoreThread(state); }
};

struct call_args {
  pd_tensor d[MAX_TENSORS];
  pd_tensor *p[MAX_TENSORS]; /* NULL where the argument is None */
  void *stream;
  int device; /* of the tensors, or -1 */
  int rc;     /* PD_OK, or the refusal of tensors that are not on one device */
};

/* The tensors args[0 .. n) and the stream of the launch (None: the current one
 * of the tensors' device). */
static bool begin(PyObject *const *args, int n, PyObject *stream, call_args *a) {
  int device = -2;
  a->rc = PD_OK;
  a->stream = nullptr;
  for (int i = 0; i < n; ++i) {
    a->p[i] = nullptr;
    if (args[i] == Py_None) continue;
    int dev;
    if (!fill(args[i], &a->d[i], &dev)) return false;
    a->p[i] = &a->d[i];
    if (device == -2) device = dev;
    if (dev != device) a->rc = PD_EINVAL;
  }
  a->device = device;
  if (a->rc != PD_OK) return true;
  if (device < 0) {
    /* host tensors: refused where there is a GPU, else left to the library,
     * which reports the missing device */
    if (c10::cuda::device_count() > 0) a->rc = PD_EINVAL;
    return true;
  }
  if (stream == Py_None) {
    a->stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    return true;
  }
  PyObject *r = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
  if (!r) return false;
  a->stream = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

/* The library's function with the tensors' device current, without the
 * interpreter's lock; its status. */
template <typename F>
static PyObject *call(call_args &a, F &&f) {
  if (a.rc == PD_OK) {
    const c10::cuda::OptionalCUDAGuard guard(
        a.device >= 0 ? std::optional<c10::Device>(c10::Device(c10::kCUDA, (c10::DeviceIndex)a.device))
                      : std::nullopt);
    const unlocked lock;
    a.rc = f();
  }
  return PyLong_FromLong(a.rc);
}

/* n integers that fit an int */
static int ints(PyObject *const *args, int n, int *out) {
  for (int i = 0; i < n; ++i) {
    const long v = PyLong_AsLong(args[i]);
    if (v == -1 && PyErr_Occurred()) return 0;
    if (v > INT32_MAX || v < INT32_MIN) {
      PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
      return 0;
    }
    out[i] = (int)v;
  }
  return 1;
}

static void *address(PyObject *o) { return o == Py_None ? NULL : PyLong_AsVoidPtr(o); }

static int counted(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
  return 0;
}

/* (q, k, v, block_table, seq_lens, query_start, out, Hq, Hkv, D, P, M,
 *  window, sinks, layout, scale, scratch, opts, stream) */
static PyObject *attn_sinks(PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[8];
  if (!counted(n, 19) || !ints(args + 7, 8, v)) return NULL;
  const float scale = (float)PyFloat_AsDouble(args[15]);
  pd_scratch *scratch = (pd_scratch *)address(args[16]);
  const pd_options *opts = (const pd_options *)address(args[17]);
  if (PyErr_Occurred() || !begin(args, 7, args[18], &a)) return NULL;
  return call(a, [&] {
    return g_attn(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], v[0], v[1], v[2], v[3],
                  v[4], v[5], v[6], scale, v[7], scratch, a.stream, opts);
  });
}

/* (q, k, v, block_table, seq_lens, query_start, work, out, Hq, Hkv, D, P,
 *  window, sinks, layout, scale, info, scratch, stream) */
static PyObject *prefill_sinks(PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[7];
  if (!counted(n, 19) || !ints(args + 8, 7, v)) return NULL;
  const float scale = (float)PyFloat_AsDouble(args[15]);
  const pd_prefill_plan_info *info = (const pd_prefill_plan_info *)address(args[16]);
  pd_scratch *scratch = (pd_scratch *)address(args[17]);
  if (PyErr_Occurred() || !begin(args, 8, args[18], &a)) return NULL;
  return call(a, [&] {
    return g_prefill(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], info, a.p[7], v[0],
                     v[1], v[2], v[3], v[4], v[5], scale, v[6], scratch, a.stream);
  });
}

/* (context_lens, query_lens, free_pages, cursor, position_delta, block_table,
 *  query_start, seq_lens, positions, slot_mapping, next_cursor, page_size,
 *  num_pages, stream) */
static PyObject *batch_tables(PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[2];
  if (!counted(n, 14) || !ints(args + 11, 2, v)) return NULL;
  if (!begin(args, 11, args[13], &a)) return NULL;
  return call(a, [&] {
    return g_tables(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], a.p[7], a.p[8],
                    a.p[9], a.p[10], v[0], v[1], a.stream);
  });
}

/* (q, k, v, positions, slot_mapping, cos_sin_cache, q_out, k_cache, v_cache,
 *  Hq, Hkv, D, rot_dim, page_size, layout, is_neox, pair_axis, stream) */
static PyObject *rope_axes(PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[7];
  if (!counted(n, 18) || !ints(args + 9, 7, v)) return NULL;
  char *pairs;
  Py_ssize_t count;
  if (PyBytes_AsStringAndSize(args[16], &pairs, &count) < 0) return NULL;
  if (count != v[3] / 2) {
    PyErr_Format(PyExc_ValueError, "pair_axis has %zd entries, rot_dim / 2 is %d", count, v[3] / 2);
    return NULL;
  }
  if (!begin(args, 9, args[17], &a)) return NULL;
  return call(a, [&] {
    return g_rope(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], (const uint8_t *)pairs, a.p[6],
                  a.p[7], a.p[8], v[0], v[1], v[2], v[3], v[4], v[5], v[6], a.stream);
  });
}

/* (q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, query_start,
 *  out, Hq, Hkv, D, P, M, window, sinks, layout, scale, scratch, stream) */
static PyObject *quant_attn(PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[8];
  if (!counted(n, 20) || !ints(args + 9, 8, v)) return NULL;
  const float scale = (float)PyFloat_AsDouble(args[17]);
  pd_scratch *scratch = (pd_scratch *)address(args[18]);
  if (PyErr_Occurred() || !begin(args, 9, args[19], &a)) return NULL;
  return call(a, [&] {
    return g_quant_attn(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], a.p[7], a.p[8],
                        v[0], v[1], v[2], v[3], v[4], v[5], v[6], scale, v[7], scratch, a.stream);
  });
}

/* (k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out_table, k_out,
 *  v_out, Hkv, D, P, layout, stream) */
static PyObject *quant_read(PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[4];
  if (!counted(n, 14) || !ints(args + 9, 4, v)) return NULL;
  if (!begin(args, 9, args[13], &a)) return NULL;
  return call(a, [&] {
    return g_quant_read(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], a.p[7], a.p[8],
                        v[0], v[1], v[2], v[3], a.stream);
  });
}

/* (q, k, v, positions, slot_mapping, cos_sin_cache, q_out, k_cache, v_cache,
 *  k_scale, v_scale, Hq, Hkv, D, rot_dim, page_size, layout, is_neox,
 *  pair_axis, stream) */
static PyObject *quant_write(PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[7];
  if (!counted(n, 20) || !ints(args + 11, 7, v)) return NULL;
  char *pairs = NULL;
  if (args[18] != Py_None) {
    Py_ssize_t count;
    if (PyBytes_AsStringAndSize(args[18], &pairs, &count) < 0) return NULL;
    if (count != v[3] / 2) {
      PyErr_Format(PyExc_ValueError, "pair_axis has %zd entries, rot_dim / 2 is %d", count,
                   v[3] / 2);
      return NULL;
    }
  }
  if (!begin(args, 11, args[19], &a)) return NULL;
  return call(a, [&] {
    return g_quant_write(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], (const uint8_t *)pairs,
                         a.p[6], a.p[7], a.p[8], a.p[9], a.p[10], v[0], v[1], v[2], v[3], v[4],
                         v[5], v[6], a.stream);
  });
}

/* setup(addresses of the seven functions) */
static PyObject *setup(PyObject *const *args, Py_ssize_t n) {
  if (!counted(n, 7)) return NULL;
  g_attn = (attn_fn)PyLong_AsVoidPtr(args[0]);
  g_prefill = (prefill_fn)PyLong_AsVoidPtr(args[1]);
  g_tables = (tables_fn)PyLong_AsVoidPtr(args[2]);
  g_rope = (rope_fn)PyLong_AsVoidPtr(args[3]);
  g_quant_attn = (quant_attn_fn)PyLong_AsVoidPtr(args[4]);
  g_quant_read = (quant_read_fn)PyLong_AsVoidPtr(args[5]);
  g_quant_write = (quant_write_fn)PyLong_AsVoidPtr(args[6]);
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

/* A method's entry: a C++ exception becomes a Python one. */
template <PyObject *(*f)(PyObject *const *, Py_ssize_t)>
static PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    return f(args, n);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return NULL;
  }
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))entry<name>, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(setup), METHOD(attn_sinks), METHOD(prefill_sinks),
                                METHOD(batch_tables), METHOD(rope_axes), METHOD(quant_attn),
                                METHOD(quant_read), METHOD(quant_write), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
