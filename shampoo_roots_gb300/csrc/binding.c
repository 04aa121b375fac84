/* Argument marshalling of the training-step operators (operators.py) in C: reads
 * what the C ABI of include/precond.h takes off torch tensors through their
 * Python attributes, and calls it.  In Python the same cost 8 us a call, twice
 * what the kernel of one token takes.  Needs neither torch's headers nor its
 * libraries; the library's entry points come from ctypes (set_up). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

typedef struct {
  void* p;
  int64_t rows, cols, ld;   /* 2-D: rows, columns, row pitch; else rows = elements, cols = ld = 1 */
  int dim, contiguous;
  PyObject* dtype;          /* borrowed: dtypes live as long as torch */
} Tensor;

enum { T_F32, T_BF16, T_E4M3, T_E8M0, T_U8, T_I32, T_I64, T_COUNT };
static PyObject* dtypes[T_COUNT];
static PyObject *s_shape, *s_stride, *s_data_ptr, *s_dtype, *s_get_device, *s_new_empty, *raw_stream;
static PyObject *raw_alloc, *raw_delete, *current_device;   /* torch's allocator, NULL where it cannot be had so */
enum { E_NORM, E_GRAD, E_GRAD_WS, E_QUANTIZE, E_GEMM, E_DISTILL, E_DISTILL_WS, E_COUNT };
static void* entry[E_COUNT];

static int bad(PyObject* type, const char* what, const char* why) {
  PyErr_Format(type, "%s %s", what, why);
  return -1;
}

/* A tensor's attributes; returns -1 with an exception set. */
static int get(PyObject* t, const char* what, Tensor* o) {
  PyObject* v = PyObject_GetAttr(t, s_shape);
  if (!v) return -1;
  if (!PyTuple_Check(v)) {
    Py_DECREF(v);
    return bad(PyExc_TypeError, what, "must be a tensor");
  }
  int64_t size[8] = {0}, step[8] = {0}, n = 1;
  o->dim = (int)PyTuple_GET_SIZE(v);
  if (o->dim > 8) {
    Py_DECREF(v);
    return bad(PyExc_ValueError, what, "has too many dimensions");
  }
  for (int i = 0; i < o->dim; ++i) {
    size[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    n *= size[i];
  }
  Py_DECREF(v);
  if (!(v = PyObject_CallMethodNoArgs(t, s_stride))) return -1;
  int64_t want = 1;
  o->contiguous = 1;
  for (int i = o->dim - 1; i >= 0; --i) {
    step[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    if (size[i] != 1 && step[i] != want && n) o->contiguous = 0;
    want *= size[i];
  }
  Py_DECREF(v);
  if (!(v = PyObject_CallMethodNoArgs(t, s_data_ptr))) return -1;
  o->p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!(v = PyObject_GetAttr(t, s_dtype))) return -1;
  o->dtype = v;
  Py_DECREF(v);
  if (PyErr_Occurred()) return -1;
  if (o->dim == 2) {
    o->rows = size[0];
    o->cols = size[1];
    if (step[1] != 1 && size[1] > 1) return bad(PyExc_ValueError, what, "must be 2-D with consecutive columns");
    o->ld = size[0] > 1 ? step[0] : (step[0] > size[1] ? step[0] : size[1]);
  } else {
    o->rows = n;
    o->cols = o->ld = 1;
  }
  return 0;
}

static int matrix(PyObject* t, const char* what, Tensor* o) {
  if (get(t, what, o)) return -1;
  return o->dim == 2 ? 0 : bad(PyExc_ValueError, what, "must be 2-D with consecutive columns");
}
static int matrix_like(PyObject* t, const char* what, Tensor* o, int64_t rows, int64_t cols, PyObject* dtype) {
  if (matrix(t, what, o)) return -1;
  if (o->rows != rows || o->cols != cols) {
    PyErr_Format(PyExc_ValueError, "%s must have shape (%lld, %lld), got (%lld, %lld)", what, (long long)rows, (long long)cols,
                 (long long)o->rows, (long long)o->cols);
    return -1;
  }
  if (dtype && o->dtype != dtype) {
    PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", what, dtype, o->dtype);
    return -1;
  }
  return 0;
}
/* An optional matrix: None leaves nulls. */
static int maybe(PyObject* t, const char* what, Tensor* o, int64_t rows, int64_t cols, PyObject* dtype) {
  o->p = NULL;
  o->ld = 0;
  return t == Py_None ? 0 : matrix_like(t, what, o, rows, cols, dtype);
}
static int vector(PyObject* t, const char* what, Tensor* o, int64_t n, int f32) {
  if (get(t, what, o)) return -1;
  if (o->dim != 1 || o->rows != n || !o->contiguous) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous vector of %lld", what, (long long)n);
    return -1;
  }
  if (f32 && o->dtype != dtypes[T_F32]) {
    PyErr_Format(PyExc_TypeError, "%s must be torch.float32, got %S", what, o->dtype);
    return -1;
  }
  return 0;
}
static int maybe_vector(PyObject* t, const char* what, Tensor* o, int64_t n) {
  o->p = NULL;
  return t == Py_None ? 0 : vector(t, what, o, n, 1);
}
/* PRECOND_F32 or PRECOND_BF16, or -1. */
static int float_type(const Tensor* t, const char* what) {
  if (t->dtype == dtypes[T_F32]) return 0;
  if (t->dtype == dtypes[T_BF16]) return 1;
  PyErr_Format(PyExc_TypeError, "%s must be float32 or bfloat16, got %S", what, t->dtype);
  return -1;
}
/* A matrix in 8-bit form; rows < 0: any shape.  A single row needs no pitch: it gets one that serves. */
static int form8(PyObject* q, PyObject* scale, const char* what, Tensor* o, Tensor* s, int64_t rows, int64_t cols) {
  if (matrix(q, what, o)) return -1;
  if (o->dtype != dtypes[T_E4M3]) {
    PyErr_Format(PyExc_TypeError, "%s must be float8_e4m3fn, got %S", what, o->dtype);
    return -1;
  }
  if (rows >= 0 && (o->rows != rows || o->cols != cols)) {
    PyErr_Format(PyExc_ValueError, "%s must have shape (%lld, %lld), got (%lld, %lld)", what, (long long)rows, (long long)cols,
                 (long long)o->rows, (long long)o->cols);
    return -1;
  }
  if (o->rows <= 1) o->ld = (o->ld + 15) / 16 * 16;
  if (scale == Py_None) return bad(PyExc_TypeError, what, "needs float8_e8m0fnu (or uint8) scales");
  if (get(scale, what, s)) return -1;
  if (s->dtype != dtypes[T_E8M0] && s->dtype != dtypes[T_U8])
    return bad(PyExc_TypeError, what, "needs float8_e8m0fnu (or uint8) scales");
  const int64_t groups = (o->cols + 511) / 512, blocks = (o->rows + 127) / 128;
  if (s->contiguous && s->rows * s->cols == groups * blocks * 512) return 0;
  PyErr_Format(PyExc_ValueError, "%s's scales must be contiguous, of shape (%lld, %lld, 32, 4, 4)", what, (long long)groups,
               (long long)blocks);
  return -1;
}
static int maybe8(PyObject* q, PyObject* scale, const char* what, Tensor* o, Tensor* s, int64_t rows, int64_t cols) {
  o->p = s->p = NULL;
  o->ld = 0;
  if (q == Py_None) return scale == Py_None ? 0 : bad(PyExc_ValueError, what, "is missing: its scales were given");
  return form8(q, scale, what, o, s, rows, cols);
}

/* The stream argument: None is torch's current stream on the tensor's device. */
static int stream_of(PyObject* stream, PyObject* t, void** out) {
  *out = NULL;
  if (stream == Py_None) {
    PyObject* d = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!d) return -1;
    if (PyLong_AsLong(d) >= 0) {
      PyObject* s = PyObject_CallOneArg(raw_stream, d);
      Py_DECREF(d);
      if (!s) return -1;
      *out = PyLong_AsVoidPtr(s);
      Py_DECREF(s);
    } else {
      Py_DECREF(d);
    }
    return PyErr_Occurred() ? -1 : 0;
  }
  if (PyLong_Check(stream)) {
    *out = PyLong_AsVoidPtr(stream);
    return PyErr_Occurred() ? -1 : 0;
  }
  PyObject* s = PyObject_GetAttrString(stream, "cuda_stream");
  if (!s) return -1;
  *out = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return PyErr_Occurred() ? -1 : 0;
}
/* The workspace argument: None is memory of torch's allocator (*own, to be given back with give_back after the call):
 * a piece of `like`'s device, or a float32 vector like it where the allocator cannot be called itself (a gradient of 45
 * x 105 takes the host 11.6 us with the vector, 6.88 with the piece).  It belongs to the current stream, so another
 * one needs a workspace of the caller's. */
static void give_back(PyObject* own) {
  if (own && PyLong_Check(own)) Py_XDECREF(PyObject_CallOneArg(raw_delete, own));
  Py_XDECREF(own);
}
static int workspace_of(PyObject* given, PyObject* like, int64_t need, PyObject* stream, void* st, Tensor* o, PyObject** own) {
  *own = NULL;
  o->p = NULL;
  o->rows = 0;
  if (given != Py_None) {
    if (get(given, "workspace", o)) return -1;
    if (o->dim != 1 || !o->contiguous || (o->dtype != dtypes[T_U8] && o->dtype != dtypes[T_F32])) {
      PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous vector of uint8 or float32");
      return -1;
    }
    if (o->dtype == dtypes[T_F32]) o->rows *= 4;
    return 0;
  }
  if (need <= 0) return 0;
  if (stream != Py_None) {
    void* current;
    if (stream_of(Py_None, like, &current)) return -1;
    if (current != st) return bad(PyExc_ValueError, "give a workspace", "with a stream other than torch's current one");
  }
  if (raw_alloc) {
    PyObject *its = PyObject_CallMethodNoArgs(like, s_get_device), *now = NULL;
    if (!its) return -1;
    const long device = PyLong_AsLong(its);
    if (device >= 0) now = PyObject_CallNoArgs(current_device);
    const int same = device < 0 ? 0 : now ? PyObject_RichCompareBool(now, its, Py_EQ) : -1;
    Py_XDECREF(now);
    Py_DECREF(its);
    if (same < 0) return -1;
    if (same) {
      PyObject *bytes = PyLong_FromLongLong(need), *where = PyLong_FromVoidPtr(st);
      if (bytes && where) *own = PyObject_CallFunctionObjArgs(raw_alloc, bytes, where, NULL);
      Py_XDECREF(bytes);
      Py_XDECREF(where);
      if (!*own) return -1;
      o->p = PyLong_AsVoidPtr(*own);
      o->rows = need;
      return 0;
    }
  }
  PyObject* n = PyLong_FromLongLong((need + 3) / 4);
  if (!n) return -1;
  *own = PyObject_CallMethodOneArg(like, s_new_empty, n);
  Py_DECREF(n);
  PyObject* p = *own ? PyObject_CallMethodNoArgs(*own, s_data_ptr) : NULL;
  if (p) {
    o->p = PyLong_AsVoidPtr(p);
    o->rows = need;
    Py_DECREF(p);
  }
  if (!PyErr_Occurred()) return 0;
  Py_CLEAR(*own);
  return -1;
}
static int handle(PyObject* h, void** out) {
  *out = h == Py_None ? NULL : PyLong_AsVoidPtr(h);
  return PyErr_Occurred() ? -1 : 0;
}
static int count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 0;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return -1;
}

/* (h, x, weight, eps, residual, total, y, q, scale, rstd, stream) */
static PyObject* rms_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, const void*, const void*, const void*, int, int, int64_t, int64_t, int64_t, int64_t, float, void*,
                    int64_t, void*, int64_t, void*, int64_t, uint8_t*, float*, void*);
  Tensor x, w, r, t, y, q, s, rs;
  void *h, *st;
  if (count(n, 11) || handle(a[0], &h) || matrix(a[1], "x", &x)) return NULL;
  const int dt = float_type(&x, "x");
  const double eps = PyFloat_AsDouble(a[3]);
  if (dt < 0 || PyErr_Occurred() || vector(a[2], "weight", &w, x.cols, 0)) return NULL;
  const int wt = float_type(&w, "weight");
  if (wt < 0 || maybe(a[4], "residual", &r, x.rows, x.cols, x.dtype) || maybe(a[5], "total", &t, x.rows, x.cols, x.dtype) ||
      maybe(a[6], "y", &y, x.rows, x.cols, x.dtype) || maybe8(a[7], a[8], "q", &q, &s, x.rows, x.cols) ||
      maybe_vector(a[9], "rstd", &rs, x.rows) || stream_of(a[10], a[1], &st))
    return NULL;
  return PyLong_FromLong(((fn)entry[E_NORM])(h, x.p, r.p, w.p, dt, wt, x.rows, x.cols, x.ld, r.ld, (float)eps, t.p, t.ld, y.p,
                                             y.ld, q.p, q.ld, s.p, rs.p, st));
}

/* (h, dy, x, weight, rstd, dx, dw, dresidual, workspace, stream) */
static PyObject* rms_norm_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, const void*, const void*, const void*, const float*, const void*, int, int, int64_t, int64_t,
                    int64_t, int64_t, int64_t, void*, int64_t, float*, void*, int64_t, void*);
  typedef int64_t (*need_fn)(int64_t, int64_t);
  PyObject* own;
  Tensor dy, x, w, rs, dx, dw, dr, ws;
  void *h, *st;
  if (count(n, 10) || handle(a[0], &h) || matrix(a[1], "dy", &dy)) return NULL;
  const int dt = float_type(&dy, "dy");
  if (dt < 0 || matrix_like(a[2], "x", &x, dy.rows, dy.cols, dy.dtype) || vector(a[3], "weight", &w, dy.cols, 0)) return NULL;
  const int wt = float_type(&w, "weight");
  if (wt < 0 || vector(a[4], "rstd", &rs, dy.rows, 1) || matrix_like(a[5], "dx", &dx, dy.rows, dy.cols, dy.dtype) ||
      vector(a[6], "dw", &dw, dy.cols, 1) || maybe(a[7], "dresidual", &dr, dy.rows, dy.cols, dy.dtype) ||
      stream_of(a[9], a[1], &st) ||
      workspace_of(a[8], a[6], a[8] == Py_None ? ((need_fn)entry[E_GRAD_WS])(dy.rows, dy.cols) : 0, a[9], st, &ws, &own))
    return NULL;
  const int code = ((fn)entry[E_GRAD])(h, dy.p, x.p, w.p, rs.p, dr.p, dt, wt, dy.rows, dy.cols, dy.ld, x.ld, dr.ld, dx.p, dx.ld,
                                       dw.p, ws.p, ws.rows, st);
  give_back(own);
  return PyErr_Occurred() ? NULL : PyLong_FromLong(code);
}

/* (h, x, q, scale, qt, scale_t, block, x_scale, stream) */
static PyObject* quantize8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, const void*, int, int64_t, int64_t, int64_t, const uint8_t*, int, void*, int64_t, uint8_t*, void*,
                    int64_t, uint8_t*, void*);
  Tensor x, xs, q, s, qt, qs;
  void *h, *st;
  if (count(n, 9) || handle(a[0], &h) || matrix(a[1], "x", &x)) return NULL;
  xs.p = NULL;
  int dt = 2;
  if (x.dtype == dtypes[T_E4M3]) {
    if (form8(a[1], a[7], "x", &x, &xs, -1, -1)) return NULL;
  } else {
    if ((dt = float_type(&x, "x")) < 0) return NULL;
    if (a[7] != Py_None) {
      PyErr_SetString(PyExc_ValueError, "x_scale goes with a float8_e4m3fn x");
      return NULL;
    }
  }
  const long block = PyLong_AsLong(a[6]);
  if (PyErr_Occurred() || maybe8(a[2], a[3], "q", &q, &s, x.rows, x.cols) || maybe8(a[4], a[5], "qt", &qt, &qs, x.cols, x.rows) ||
      stream_of(a[8], a[1], &st))
    return NULL;
  return PyLong_FromLong(((fn)entry[E_QUANTIZE])(h, x.p, dt, x.rows, x.cols, x.ld, xs.p, (int)block, q.p, q.ld, s.p, qt.p, qt.ld,
                                                 qs.p, st));
}

/* (h, a, scale_a, b, scale_b, out, accumulate, stream) */
static PyObject* gemm8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, int64_t, int64_t, int64_t, const void*, int64_t, const uint8_t*, const void*, int64_t, const uint8_t*,
                    void*, int64_t, int, int, void*);
  Tensor A, sa, B, sb, c;
  void *h, *st;
  if (count(n, 8) || handle(a[0], &h) || form8(a[1], a[2], "a", &A, &sa, -1, -1) ||
      form8(a[3], a[4], "b", &B, &sb, -1, -1))
    return NULL;
  if (A.cols != B.cols) {
    PyErr_Format(PyExc_ValueError, "a and b must have the same number of columns, got %lld and %lld", (long long)A.cols,
                 (long long)B.cols);
    return NULL;
  }
  if (matrix_like(a[5], "out", &c, A.rows, B.rows, NULL)) return NULL;
  const int ct = float_type(&c, "out");
  const int acc = PyObject_IsTrue(a[6]);
  if (ct < 0 || acc < 0 || stream_of(a[7], a[5], &st)) return NULL;
  return PyLong_FromLong(((fn)entry[E_GEMM])(h, A.rows, B.rows, A.cols, A.p, A.ld, sa.p, B.p, B.ld, sb.p, c.p, c.ld, ct, acc, st));
}

/* (h, logits, ids, teacher, loss, weight, temperature, dlogits, workspace, stream) */
static PyObject* distill(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, const void*, int, int64_t, int64_t, int64_t, const void*, int, int64_t, const void*, int, int64_t, int,
                    const float*, float, float*, void*, int64_t, void*, int64_t, void*);
  typedef int64_t (*need_fn)(int64_t, int64_t, int, int, int);
  PyObject* own;
  Tensor z, ids, t, loss, w, dz, ws;
  void *h, *st;
  if (count(n, 10) || handle(a[0], &h) || matrix(a[1], "logits", &z)) return NULL;
  const int dt = float_type(&z, "logits");
  if (dt < 0 || matrix(a[2], "ids", &ids)) return NULL;
  if (ids.dtype != dtypes[T_I32] && ids.dtype != dtypes[T_I64]) {
    PyErr_Format(PyExc_TypeError, "ids must be int32 or int64, got %S", ids.dtype);
    return NULL;
  }
  if (matrix_like(a[2], "ids", &ids, z.rows, ids.cols, NULL) || matrix_like(a[3], "teacher", &t, z.rows, ids.cols, NULL)) return NULL;
  const int tt = float_type(&t, "teacher");
  const double tau = PyFloat_AsDouble(a[6]);
  if (tt < 0 || PyErr_Occurred() || vector(a[4], "loss", &loss, z.rows, 1) || maybe_vector(a[5], "weight", &w, z.rows) ||
      maybe(a[7], "dlogits", &dz, z.rows, z.cols, z.dtype) || stream_of(a[9], a[1], &st))
    return NULL;
  const int top = (int)(ids.cols > 1 << 30 ? 1 << 30 : ids.cols);
  if (workspace_of(a[8], a[4], a[8] == Py_None ? ((need_fn)entry[E_DISTILL_WS])(z.rows, z.cols, top, dt, dz.p == z.p) : 0, a[9], st,
                   &ws, &own))
    return NULL;
  const int code = ((fn)entry[E_DISTILL])(h, z.p, dt, z.rows, z.cols, z.ld, ids.p, ids.dtype == dtypes[T_I32] ? 32 : 64, ids.ld, t.p,
                                          tt, t.ld, top, w.p, (float)tau, loss.p, dz.p, dz.ld, ws.p, ws.rows, st);
  give_back(own);
  return PyErr_Occurred() ? NULL : PyLong_FromLong(code);
}

/* set_up(dtypes, raw_stream, entries, (raw_alloc, raw_delete, current_device) or None): what the calls need, once. */
static PyObject* set_up(PyObject* self, PyObject* args) {
  PyObject *types, *raw, *addresses, *allocator;
  if (!PyArg_ParseTuple(args, "O!OO!O", &PyTuple_Type, &types, &raw, &PyTuple_Type, &addresses, &allocator)) return NULL;
  if (allocator != Py_None && (!PyArg_ParseTuple(allocator, "OOO", &raw_alloc, &raw_delete, &current_device))) return NULL;
  Py_XINCREF(raw_alloc);
  Py_XINCREF(raw_delete);
  Py_XINCREF(current_device);
  if (PyTuple_GET_SIZE(types) != T_COUNT || PyTuple_GET_SIZE(addresses) != E_COUNT) {
    PyErr_SetString(PyExc_ValueError, "wrong number of dtypes or entries");
    return NULL;
  }
  for (int i = 0; i < E_COUNT; ++i) entry[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
  if (PyErr_Occurred()) return NULL;
  for (int i = 0; i < T_COUNT; ++i) {
    dtypes[i] = PyTuple_GET_ITEM(types, i);
    Py_INCREF(dtypes[i]);
  }
  raw_stream = raw;
  Py_INCREF(raw);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"set_up", set_up, METH_VARARGS, NULL},
    {"rms_norm", (PyCFunction)(void (*)(void))rms_norm, METH_FASTCALL, NULL},
    {"rms_norm_grad", (PyCFunction)(void (*)(void))rms_norm_grad, METH_FASTCALL, NULL},
    {"quantize8", (PyCFunction)(void (*)(void))quantize8, METH_FASTCALL, NULL},
    {"gemm8", (PyCFunction)(void (*)(void))gemm8, METH_FASTCALL, NULL},
    {"distill", (PyCFunction)(void (*)(void))distill, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods};

PyMODINIT_FUNC PyInit__binding(void) {
  if (!(s_shape = PyUnicode_InternFromString("shape")) || !(s_stride = PyUnicode_InternFromString("stride")) ||
      !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) || !(s_dtype = PyUnicode_InternFromString("dtype")) ||
      !(s_get_device = PyUnicode_InternFromString("get_device")) || !(s_new_empty = PyUnicode_InternFromString("new_empty")))
    return NULL;
  return PyModule_Create(&module);
}
