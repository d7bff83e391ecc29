/*
 * Argument marshalling of the norm and expert calls for Python.
 *
 * A decode step's kernels last a few microseconds; describing eight tensors
 * to ctypes from Python takes as long.  These functions read the tensors'
 * attributes through the C API, check them as the binding's Python code does
 * for the other calls, and call the library.  They return its status.  Nothing
 * is kept between calls.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "aal.h"

typedef aal_status (*norm_fwd_fn)(aal_mat, aal_mat, aal_mat, aal_mat, float, aal_mat, aal_mat, float*, float*, void*);
typedef aal_status (*norm_bwd_fn)(aal_mat, aal_mat, const float*, const float*, aal_mat, aal_mat, aal_mat, aal_mat,
                                  aal_mat, int32_t, void*);
typedef aal_status (*moe_fn)(int32_t, int32_t, const int64_t*, aal_mat, aal_mat, aal_mat, aal_mat, aal_mat, aal_mat,
                             int32_t, int32_t, int32_t*, float*, aal_mat, aal_mat, void*);

static norm_fwd_fn f_norm_fwd;
static norm_bwd_fn f_norm_bwd;
static moe_fn f_moe;
static PyObject *d_bf16, *d_f32, *d_i32, *d_i64;   /* torch dtypes */
static PyObject *py_device, *py_stream;            /* current device; raw stream of a device */
static PyObject *s_data_ptr, *s_shape, *s_stride, *s_dtype, *s_get_device, *s_numel, *s_is_contiguous;

/* Device of the call: kNone until a tensor with entries has been seen (a host
 * tensor says -1). */
enum { kNone = -2 };
typedef struct {
  long dev;
} call_ctx;

static int long_of(PyObject* o, long long* out) { /* steals o */
  if (!o) return -1;
  *out = PyLong_AsLongLong(o);
  Py_DECREF(o);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}
static int call_long(PyObject* t, PyObject* name, long long* out) {
  return long_of(PyObject_CallMethodNoArgs(t, name), out);
}

static int place(call_ctx* c, PyObject* t, void** ptr) {
  long long dev, p;
  if (call_long(t, s_get_device, &dev)) return -1;
  if (dev != c->dev) {
    if (dev < 0) {
      PyErr_SetString(PyExc_ValueError, "tensor must be on a CUDA device");
      return -1;
    }
    if (c->dev >= 0) {
      PyErr_Format(PyExc_ValueError, "tensor is on CUDA device %lld, the current one is %ld", dev, c->dev);
      return -1;
    }
    long long cur;
    if (long_of(PyObject_CallNoArgs(py_device), &cur)) return -1;
    if (dev != cur) {
      PyErr_Format(PyExc_ValueError, "tensor is on CUDA device %lld, the current one is %lld", dev, cur);
      return -1;
    }
    c->dev = (long)dev;
  }
  PyObject* o = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!o) return -1;
  p = (long long)PyLong_AsUnsignedLongLong(o);
  Py_DECREF(o);
  if (p == -1 && PyErr_Occurred()) return -1;
  *ptr = (void*)(uintptr_t)p;
  return 0;
}

/* 1: not a dtype of a matrix */
static int dtype_code(PyObject* t, int32_t* code) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return -1;
  const int rc = d == d_bf16 ? (*code = AAL_BF16, 0) : d == d_f32 ? (*code = AAL_F32, 0) : 1;
  if (rc == 1) PyErr_Format(PyExc_ValueError, "unsupported dtype %S", d);
  Py_DECREF(d);
  return rc;
}

static int pair_of(PyObject* tuple, long long* a, long long* b) { /* steals tuple; 1: not two entries */
  if (!tuple) return -1;
  int rc = 1;
  if (PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == 2) {
    *a = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, 0));
    *b = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, 1));
    rc = PyErr_Occurred() ? -1 : 0;
  }
  Py_DECREF(tuple);
  return rc;
}

static int get_mat(call_ctx* c, PyObject* t, aal_mat* m) {
  m->ptr = NULL;
  m->dtype = AAL_BF16;
  m->rows = m->cols = m->ld = 0;
  if (t == Py_None) return 0;
  if (dtype_code(t, &m->dtype)) return -1;
  long long rows, cols, ld, unit;
  int rc = pair_of(PyObject_GetAttr(t, s_shape), &rows, &cols);
  if (rc) {
    if (rc == 1) PyErr_SetString(PyExc_ValueError, "expected a 2-D tensor");
    return -1;
  }
  m->rows = rows;
  m->cols = m->ld = cols;
  if (!rows || !cols) return 0;
  if (pair_of(PyObject_CallMethodNoArgs(t, s_stride), &ld, &unit)) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "expected a 2-D tensor");
    return -1;
  }
  if (unit != 1 && cols > 1) {
    PyErr_SetString(PyExc_ValueError, "tensor must be row-major (unit column stride)");
    return -1;
  }
  if (rows > 1) {
    if (ld < cols) {
      PyErr_SetString(PyExc_ValueError, "the rows of a tensor must not overlap");
      return -1;
    }
    m->ld = ld;
  }
  return place(c, t, &m->ptr);
}

static int contiguous(PyObject* t) {
  PyObject* o = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!o) return -1;
  const int yes = o == Py_True;
  Py_DECREF(o);
  return yes;
}

static int get_vec(call_ctx* c, PyObject* t, const char* what, aal_mat* m) {
  m->ptr = NULL;
  m->dtype = AAL_BF16;
  m->rows = m->cols = m->ld = 0;
  if (t == Py_None) return 0;
  PyObject* shape = PyObject_GetAttr(t, s_shape);
  if (!shape) return -1;
  const int one = PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 1;
  const long long n = one ? PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0)) : 0;
  Py_DECREF(shape);
  if (!one) {
    PyErr_Format(PyExc_ValueError, "%s must be 1-D", what);
    return -1;
  }
  const int cont = contiguous(t);
  if (cont < 0) return -1;
  const int rc = dtype_code(t, &m->dtype);
  if (rc < 0) return -1;
  if (rc || !cont) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous, bf16 or fp32", what);
    return -1;
  }
  m->rows = 1;
  m->cols = m->ld = n;
  return n ? place(c, t, &m->ptr) : 0;
}

static int get_array(call_ctx* c, PyObject* t, PyObject* dtype, long long n, const char* what, void** ptr) {
  *ptr = NULL;
  if (t == Py_None) return 0;
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return -1;
  Py_DECREF(d); /* (dtypes are immortal singletons) */
  if (d != dtype) {
    PyErr_Format(PyExc_ValueError, "%s must be %S", what, dtype);
    return -1;
  }
  long long have;
  if (call_long(t, s_numel, &have)) return -1;
  const int cont = contiguous(t);
  if (cont < 0) return -1;
  if (have != n || !cont) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous with %lld entries", what, n);
    return -1;
  }
  return n ? place(c, t, ptr) : 0;
}

/* An argument that may be left out must not pass for left out by being empty. */
static int not_empty(PyObject* t, const aal_mat* m, const char* what) {
  if (t == Py_None || m->ptr) return 0;
  PyErr_Format(PyExc_ValueError, "%s has no entries: its shape must be that of the call", what);
  return -1;
}

/* The stream handed in, or the current one of the call's device. */
static int get_stream(const call_ctx* c, PyObject* given, void** out) {
  *out = NULL;
  PyObject* o;
  if (given != Py_None) {
    o = given;
    Py_INCREF(o);
  } else {
    if (c->dev < 0) return 0; /* nothing to launch */
    PyObject* dev = PyLong_FromLong(c->dev);
    if (!dev) return -1;
    o = PyObject_CallOneArg(py_stream, dev);
    Py_DECREF(dev);
    if (!o) return -1;
  }
  *out = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(o);
  Py_DECREF(o);
  return PyErr_Occurred() ? -1 : 0;
}

static int ready(Py_ssize_t n, Py_ssize_t want, const void* fn) {
  if (n == want && fn) return 1;
  PyErr_SetString(PyExc_TypeError, fn ? "wrong number of arguments" : "setup() has not been called");
  return 0;
}

/* Returns the library call's status.  Other threads run meanwhile: a launch may
 * wait for room in the stream's queue, or for a kernel to be loaded.  (The
 * tensors stay alive: the caller's arguments hold them.) */
#define CALL(call)                  \
  do {                              \
    aal_status status;              \
    Py_BEGIN_ALLOW_THREADS          \
    status = call;                  \
    Py_END_ALLOW_THREADS            \
    return PyLong_FromLong(status); \
  } while (0)

/* (X, gamma, beta, Y, eps, R, S, mean, rstd, stream) */
static PyObject* norm_fwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  call_ctx c = {kNone};
  aal_mat X, R, g, b, S, Y;
  void *mean, *rstd, *stream;
  if (!ready(n, 10, (const void*)f_norm_fwd)) return NULL;
  if (get_mat(&c, a[0], &X) || get_mat(&c, a[5], &R) || get_vec(&c, a[1], "gamma", &g) ||
      get_vec(&c, a[2], "beta", &b) || get_mat(&c, a[6], &S) || get_mat(&c, a[3], &Y) ||
      get_array(&c, a[7], d_f32, X.rows, "mean", &mean) || get_array(&c, a[8], d_f32, X.rows, "rstd", &rstd) ||
      get_stream(&c, a[9], &stream))
    return NULL;
  if (X.ptr && (not_empty(a[5], &R, "R") || not_empty(a[1], &g, "gamma") || not_empty(a[2], &b, "beta") ||
                not_empty(a[6], &S, "S")))
    return NULL;
  const double eps = PyFloat_AsDouble(a[4]);
  if (eps == -1.0 && PyErr_Occurred()) return NULL;
  CALL(f_norm_fwd(X, R, g, b, (float)eps, S, Y, (float*)mean, (float*)rstd, stream));
}

/* (X, gamma, mean, rstd, dY, dX, dgamma, dbeta, dR, accumulate, stream) */
static PyObject* norm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  call_ctx c = {kNone};
  aal_mat X, g, dY, dR, dX, dg, db;
  void *mean, *rstd, *stream;
  if (!ready(n, 11, (const void*)f_norm_bwd)) return NULL;
  const int acc = PyObject_IsTrue(a[9]);
  if (acc < 0 || get_mat(&c, a[0], &X) || get_vec(&c, a[1], "gamma", &g) || get_mat(&c, a[4], &dY) ||
      get_mat(&c, a[8], &dR) || get_mat(&c, a[5], &dX) || get_vec(&c, a[6], "dgamma", &dg) ||
      get_vec(&c, a[7], "dbeta", &db) || get_array(&c, a[2], d_f32, X.rows, "mean", &mean) ||
      get_array(&c, a[3], d_f32, X.rows, "rstd", &rstd) || get_stream(&c, a[10], &stream))
    return NULL;
  if (X.cols && (not_empty(a[1], &g, "gamma") || not_empty(a[6], &dg, "dgamma") || not_empty(a[7], &db, "dbeta")))
    return NULL;
  if (X.ptr && (not_empty(a[8], &dR, "dR") || not_empty(a[5], &dX, "dX"))) return NULL;
  CALL(f_norm_bwd(X, g, (const float*)mean, (const float*)rstd, dY, dR, dX, dg, db, acc, stream));
}

/* (law, q, positions, x, Wr, Wg, Wu, Wd, ids, weights, h, y, R, renormalize, stream) */
static PyObject* moe(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  call_ctx c = {kNone};
  aal_mat x, wr, wg, wu, wd, r, h, y;
  void *pos, *ids, *wt, *stream;
  if (!ready(n, 15, (const void*)f_moe)) return NULL;
  const long law = PyLong_AsLong(a[0]), q = PyLong_AsLong(a[1]);
  if (PyErr_Occurred()) return NULL;
  const int renorm = PyObject_IsTrue(a[13]);
  long long rows, k;
  if (renorm < 0 || get_mat(&c, a[3], &x)) return NULL;
  int rc = pair_of(PyObject_GetAttr(a[8], s_shape), &rows, &k);
  if (rc < 0) return NULL;
  if (rc || rows != x.rows || k > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "ids must be [entries, top_k]");
    return NULL;
  }
  if (law != (int32_t)law || q != (int32_t)q) {
    PyErr_SetString(PyExc_ValueError, "law and q must be 32-bit integers");
    return NULL;
  }
  if (get_array(&c, a[2], d_i64, rows, "positions", &pos) || get_mat(&c, a[4], &wr) || get_mat(&c, a[5], &wg) ||
      get_mat(&c, a[6], &wu) || get_mat(&c, a[7], &wd) || get_mat(&c, a[12], &r) || get_mat(&c, a[10], &h) ||
      get_mat(&c, a[11], &y) || get_array(&c, a[8], d_i32, rows * k, "ids", &ids) ||
      get_array(&c, a[9], d_f32, rows * k, "weights", &wt) || get_stream(&c, a[14], &stream))
    return NULL;
  if (x.ptr && not_empty(a[12], &r, "R")) return NULL;
  CALL(f_moe((int32_t)law, (int32_t)q, (const int64_t*)pos, x, wr, wg, wu, wd, r, (int32_t)k, renorm, (int32_t*)ids,
             (float*)wt, h, y, stream));
}

/* (addresses of the three calls; torch.bfloat16, float32, int32, int64; the
 * current device's and a device's raw stream's functions) */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!ready(n, 9, (const void*)setup)) return NULL;
  void* f[3];
  for (int i = 0; i < 3; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return NULL;
  PyObject** keep[6] = {&d_bf16, &d_f32, &d_i32, &d_i64, &py_device, &py_stream};
  for (int i = 0; i < 6; ++i) {
    Py_INCREF(a[3 + i]);
    Py_XSETREF(*keep[i], a[3 + i]);
  }
  f_norm_fwd = (norm_fwd_fn)f[0];
  f_norm_bwd = (norm_bwd_fn)f[1];
  f_moe = (moe_fn)f[2];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
                                {"layer_norm_fwd", (PyCFunction)(void (*)(void))norm_fwd, METH_FASTCALL, NULL},
                                {"layer_norm_bwd", (PyCFunction)(void (*)(void))norm_bwd, METH_FASTCALL, NULL},
                                {"moe_decode", (PyCFunction)(void (*)(void))moe, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
  struct {
    PyObject** at;
    const char* name;
  } names[] = {{&s_data_ptr, "data_ptr"}, {&s_shape, "shape"}, {&s_stride, "stride"}, {&s_dtype, "dtype"},
               {&s_get_device, "get_device"}, {&s_numel, "numel"}, {&s_is_contiguous, "is_contiguous"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].at = PyUnicode_InternFromString(names[i].name))) return NULL;
  return PyModule_Create(&module);
}
