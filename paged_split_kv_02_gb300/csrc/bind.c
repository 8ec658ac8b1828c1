/* Argument marshalling of the calls of paged_step.h: tensors to descriptors,
 * the launch's device and stream, then the library's function.  A serving
 * step makes these calls between kernels of a few microseconds each; filling
 * ctypes structures in Python took 18-20 us a call on the host of a GB300,
 * more than most of the kernels.  Nothing is computed here. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "paged_step.h"

#define MAX_TENSORS 12

static PyObject *s_data_ptr, *s_dtype, *s_shape, *s_stride, *s_get_device, *s_cuda_stream;
/* dtype objects and their codes; callables of torch */
static PyObject *g_dtypes, *g_raw_stream, *g_current, *g_set_device, *g_available;

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
static attn_fn g_attn;
static prefill_fn g_prefill;
static tables_fn g_tables;
static rope_fn g_rope;

/* The descriptor of a tensor; its device index (-1: not CUDA) in *device. */
static int fill(PyObject *t, pd_tensor *d, long *device) {
  int ok = 0;
  PyObject *ptr = NULL, *dtype = NULL, *shape = NULL, *stride = NULL, *dev = NULL;
  if (!(ptr = PyObject_CallMethodNoArgs(t, s_data_ptr))) goto done;
  if (!(dtype = PyObject_GetAttr(t, s_dtype))) goto done;
  if (!(shape = PyObject_GetAttr(t, s_shape))) goto done;
  if (!(stride = PyObject_CallMethodNoArgs(t, s_stride))) goto done;
  if (!(dev = PyObject_CallMethodNoArgs(t, s_get_device))) goto done;
  if (!PyTuple_Check(shape) || !PyTuple_Check(stride)) {
    PyErr_SetString(PyExc_TypeError, "a tensor's shape and strides are tuples");
    goto done;
  }
  memset(d, 0, sizeof *d);
  d->data = PyLong_AsVoidPtr(ptr);
  PyObject *code = PyDict_GetItemWithError(g_dtypes, dtype);
  if (!code && PyErr_Occurred()) goto done;
  d->dtype = code ? (int32_t)PyLong_AsLong(code) : 99; /* a type the library does not take */
  const Py_ssize_t n = PyTuple_GET_SIZE(shape);
  if (PyTuple_GET_SIZE(stride) != n) {
    PyErr_SetString(PyExc_TypeError, "a tensor has as many strides as dimensions");
    goto done;
  }
  d->ndim = (int32_t)n;
  for (Py_ssize_t i = 0; i < n && i < 4; ++i) {
    d->shape[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    d->stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, i));
  }
  *device = PyLong_AsLong(dev);
  ok = !PyErr_Occurred();
done:
  Py_XDECREF(ptr);
  Py_XDECREF(dtype);
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  Py_XDECREF(dev);
  return ok;
}

typedef struct {
  pd_tensor d[MAX_TENSORS];
  pd_tensor *p[MAX_TENSORS]; /* NULL where the argument is None */
  void *stream;
  long restore; /* device to make current again, or -1 */
  int rc;       /* PD_OK, or the refusal of tensors that are not on one device */
} call_args;

/* The tensors args[0 .. n), the stream of the launch (None: the current one
 * of the tensors' device), and that device made current. */
static int begin(PyObject *const *args, int n, PyObject *stream, call_args *a) {
  long device = -2;
  a->restore = -1;
  a->rc = PD_OK;
  a->stream = NULL;
  for (int i = 0; i < n; ++i) {
    a->p[i] = NULL;
    if (args[i] == Py_None) continue;
    long dev;
    if (!fill(args[i], &a->d[i], &dev)) return 0;
    a->p[i] = &a->d[i];
    if (device == -2) device = dev;
    if (dev != device) a->rc = PD_EINVAL;
  }
  if (a->rc != PD_OK) return 1;
  if (device < 0) {
    /* host tensors: refused where there is a GPU, else left to the library,
     * which reports the missing device */
    PyObject *there = PyObject_CallNoArgs(g_available);
    if (!there) return 0;
    if (PyObject_IsTrue(there)) a->rc = PD_EINVAL;
    Py_DECREF(there);
    return 1;
  }
  PyObject *index = PyLong_FromLong(device), *r;
  if (!index) return 0;
  if (stream == Py_None) {
    r = PyObject_CallOneArg(g_raw_stream, index);
  } else if (PyLong_Check(stream)) {
    r = Py_NewRef(stream);
  } else {
    r = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (r) {
    a->stream = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
  }
  r = PyErr_Occurred() ? NULL : PyObject_CallNoArgs(g_current);
  if (r) {
    const long current = PyLong_AsLong(r);
    Py_DECREF(r);
    if (current != device && !PyErr_Occurred()) {
      r = PyObject_CallOneArg(g_set_device, index);
      if (r) a->restore = current;
      Py_XDECREF(r);
    }
  }
  Py_DECREF(index);
  return !PyErr_Occurred();
}

static PyObject *end(call_args *a) {
  if (a->restore >= 0) {
    PyObject *index = PyLong_FromLong(a->restore);
    PyObject *r = index ? PyObject_CallOneArg(g_set_device, index) : NULL;
    Py_XDECREF(index);
    if (!r) return NULL;
    Py_DECREF(r);
  }
  return PyLong_FromLong(a->rc);
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

#define CALL(a, expr)        \
  if ((a).rc == PD_OK) {     \
    Py_BEGIN_ALLOW_THREADS   \
    (a).rc = (expr);         \
    Py_END_ALLOW_THREADS     \
  }

/* (q, k, v, block_table, seq_lens, query_start, out, Hq, Hkv, D, P, M,
 *  window, sinks, layout, scale, scratch, opts, stream) */
static PyObject *attn_sinks(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[8];
  (void)self;
  if (!counted(n, 19) || !ints(args + 7, 8, v)) return NULL;
  const float scale = (float)PyFloat_AsDouble(args[15]);
  pd_scratch *scratch = address(args[16]);
  const pd_options *opts = address(args[17]);
  if (PyErr_Occurred() || !begin(args, 7, args[18], &a)) return NULL;
  CALL(a, g_attn(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], v[0], v[1], v[2], v[3],
                 v[4], v[5], v[6], scale, v[7], scratch, a.stream, opts))
  return end(&a);
}

/* (q, k, v, block_table, seq_lens, query_start, work, out, Hq, Hkv, D, P,
 *  window, sinks, layout, scale, info, scratch, stream) */
static PyObject *prefill_sinks(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[7];
  (void)self;
  if (!counted(n, 19) || !ints(args + 8, 7, v)) return NULL;
  const float scale = (float)PyFloat_AsDouble(args[15]);
  const pd_prefill_plan_info *info = address(args[16]);
  pd_scratch *scratch = address(args[17]);
  if (PyErr_Occurred() || !begin(args, 8, args[18], &a)) return NULL;
  CALL(a, g_prefill(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], info, a.p[7], v[0],
                    v[1], v[2], v[3], v[4], v[5], scale, v[6], scratch, a.stream))
  return end(&a);
}

/* (context_lens, query_lens, free_pages, cursor, position_delta, block_table,
 *  query_start, seq_lens, positions, slot_mapping, next_cursor, page_size,
 *  num_pages, stream) */
static PyObject *batch_tables(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[2];
  (void)self;
  if (!counted(n, 14) || !ints(args + 11, 2, v)) return NULL;
  if (!begin(args, 11, args[13], &a)) return NULL;
  CALL(a, g_tables(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], a.p[7], a.p[8], a.p[9],
                   a.p[10], v[0], v[1], a.stream))
  return end(&a);
}

/* (q, k, v, positions, slot_mapping, cos_sin_cache, q_out, k_cache, v_cache,
 *  Hq, Hkv, D, rot_dim, page_size, layout, is_neox, pair_axis, stream) */
static PyObject *rope_axes(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  call_args a;
  int v[7];
  (void)self;
  if (!counted(n, 18) || !ints(args + 9, 7, v)) return NULL;
  char *pairs;
  Py_ssize_t count;
  if (PyBytes_AsStringAndSize(args[16], &pairs, &count) < 0) return NULL;
  if (count != v[3] / 2) {
    PyErr_Format(PyExc_ValueError, "pair_axis has %zd entries, rot_dim / 2 is %d", count, v[3] / 2);
    return NULL;
  }
  if (!begin(args, 9, args[17], &a)) return NULL;
  CALL(a, g_rope(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], (const uint8_t *)pairs, a.p[6],
                 a.p[7], a.p[8], v[0], v[1], v[2], v[3], v[4], v[5], v[6], a.stream))
  return end(&a);
}

/* setup(addresses of the four functions, dtype codes, current raw stream of a
 * device, current device, set device, whether CUDA is available) */
static PyObject *setup(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  (void)self;
  if (!counted(n, 9)) return NULL;
  g_attn = (attn_fn)PyLong_AsVoidPtr(args[0]);
  g_prefill = (prefill_fn)PyLong_AsVoidPtr(args[1]);
  g_tables = (tables_fn)PyLong_AsVoidPtr(args[2]);
  g_rope = (rope_fn)PyLong_AsVoidPtr(args[3]);
  if (PyErr_Occurred()) return NULL;
  if (!PyDict_Check(args[4])) {
    PyErr_SetString(PyExc_TypeError, "the dtype codes are a dict");
    return NULL;
  }
  PyObject **to[] = {&g_dtypes, &g_raw_stream, &g_current, &g_set_device, &g_available};
  for (int i = 0; i < 5; ++i) Py_XSETREF(*to[i], Py_NewRef(args[4 + i]));
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(setup), METHOD(attn_sinks), METHOD(prefill_sinks),
                                METHOD(batch_tables), METHOD(rope_axes), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__bind(void) {
  PyObject **names[] = {&s_data_ptr, &s_dtype, &s_shape, &s_stride, &s_get_device, &s_cuda_stream};
  const char *text[] = {"data_ptr", "dtype", "shape", "stride", "get_device", "cuda_stream"};
  for (int i = 0; i < 6; ++i)
    if (!(*names[i] = PyUnicode_InternFromString(text[i]))) return NULL;
  return PyModule_Create(&module);
}
