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
  int dim, contiguous, dense;   /* dense: consecutive elements, in whatever order */
  PyObject* dtype;          /* borrowed: dtypes live as long as torch */
} Tensor;

enum { T_F32, T_BF16, T_E4M3, T_E8M0, T_U8, T_I32, T_I64, T_COUNT };
static PyObject* dtypes[T_COUNT];
static PyObject *s_shape, *s_stride, *s_is_contiguous, *s_data_ptr, *s_dtype, *s_get_device, *s_new_empty, *raw_stream;
static PyObject *raw_alloc, *raw_delete, *current_device;   /* torch's allocator, NULL where it cannot be had so */
enum { E_NORM, E_GRAD, E_GRAD_WS, E_QUANTIZE, E_GEMM, E_DISTILL, E_DISTILL_WS, E_LAYER, E_LAYER_GRAD, E_LAYER_GRAD_WS, E_POLICY,
       E_LIST, E_LIST_END, E_LIST_WS, E_GRAD_NORM, E_CLIP, E_COUNT };
static void* entry[E_COUNT];

static int bad(PyObject* type, const char* what, const char* why) {
  PyErr_Format(type, "%s %s", what, why);
  return -1;
}

/* A tensor's attributes; returns -1 with an exception set.  (`any`: of any strides, as a run of elements.) */
static int get_as(PyObject* t, const char* what, Tensor* o, int any) {
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
  o->contiguous = 0;
  if (o->dim != 2 || any) {     /* the strides themselves are asked for where they count: of matrices, and of what has gaps */
    if (!(v = PyObject_CallMethodNoArgs(t, s_is_contiguous))) return -1;
    o->contiguous = v == Py_True;
    Py_DECREF(v);
  }
  o->dense = o->contiguous;
  if (!o->contiguous && (o->dim == 2 || any)) {
    if (!(v = PyObject_CallMethodNoArgs(t, s_stride))) return -1;
    for (int i = 0; i < o->dim; ++i) step[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    Py_DECREF(v);
    int used = 0;               /* the dimensions by their strides: each as long as those within it */
    int64_t inner = 1;
    for (int found = any; found;) {
      found = 0;
      for (int i = 0; i < o->dim; ++i)
        if (!(used >> i & 1) && size[i] != 1 && step[i] == inner) {
          used |= 1 << i;
          inner *= size[i];
          found = 1;
        }
    }
    o->dense = any && inner == n;
    if (!any)
      o->contiguous = o->dense = n == 0 || ((size[1] == 1 || step[1] == 1) && (size[0] == 1 || step[0] == size[1]));
  }
  if (!(v = PyObject_CallMethodNoArgs(t, s_data_ptr))) return -1;
  o->p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!(v = PyObject_GetAttr(t, s_dtype))) return -1;
  o->dtype = v;
  Py_DECREF(v);
  if (PyErr_Occurred()) return -1;
  if (o->dim == 2 && !any) {
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
static int get(PyObject* t, const char* what, Tensor* o) { return get_as(t, what, o, 0); }

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
/* All tensors among the n arguments are on one device. */
static int one_device(PyObject* const* a, Py_ssize_t n) {
  long device = 0;
  int seen = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (a[i] == Py_None) continue;
    PyObject* d = PyObject_CallMethodNoArgs(a[i], s_get_device);
    if (!d) return -1;
    const long its = PyLong_AsLong(d);
    Py_DECREF(d);
    if (its == -1 && PyErr_Occurred()) return -1;
    if (seen && its != device) {
      PyErr_SetString(PyExc_ValueError, "the tensors must be on one device");
      return -1;
    }
    device = its;
    seen = 1;
  }
  return 0;
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

/* (h, x, weight, eps, bias, residual, total, y, q, scale, mean, rstd, stream) */
static PyObject* layer_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, const void*, const void*, const void*, const void*, int, int, int64_t, int64_t, int64_t, int64_t, float,
                    void*, int64_t, void*, int64_t, void*, int64_t, uint8_t*, float*, float*, void*);
  Tensor x, w, b, r, t, y, q, s, m, rs;
  void *h, *st;
  if (count(n, 13) || handle(a[0], &h) || matrix(a[1], "x", &x)) return NULL;
  const int dt = float_type(&x, "x");
  const double eps = PyFloat_AsDouble(a[3]);
  if (dt < 0 || PyErr_Occurred() || vector(a[2], "weight", &w, x.cols, 0)) return NULL;
  const int wt = float_type(&w, "weight");
  if (wt < 0) return NULL;
  b.p = NULL;
  if (a[4] != Py_None) {
    if (vector(a[4], "bias", &b, x.cols, 0)) return NULL;
    if (b.dtype != w.dtype) {
      PyErr_Format(PyExc_TypeError, "bias must be %S, as weight is, got %S", w.dtype, b.dtype);
      return NULL;
    }
  }
  if (maybe(a[5], "residual", &r, x.rows, x.cols, x.dtype) || maybe(a[6], "total", &t, x.rows, x.cols, x.dtype) ||
      maybe(a[7], "y", &y, x.rows, x.cols, x.dtype) || maybe8(a[8], a[9], "q", &q, &s, x.rows, x.cols) ||
      maybe_vector(a[10], "mean", &m, x.rows) || maybe_vector(a[11], "rstd", &rs, x.rows))
    return NULL;
  PyObject* tensors[10] = {a[1], a[2], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11]};
  if (one_device(tensors, 10) || stream_of(a[12], a[1], &st)) return NULL;
  return PyLong_FromLong(((fn)entry[E_LAYER])(h, x.p, r.p, w.p, b.p, dt, wt, x.rows, x.cols, x.ld, r.ld, (float)eps, t.p, t.ld, y.p,
                                              y.ld, q.p, q.ld, s.p, m.p, rs.p, st));
}

/* (h, dy, x, weight, mean, rstd, dx, dw, db, dresidual, workspace, stream) */
static PyObject* layer_norm_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, const void*, const void*, const void*, const float*, const float*, const void*, int, int, int64_t, int64_t,
                    int64_t, int64_t, int64_t, void*, int64_t, float*, float*, void*, int64_t, void*);
  typedef int64_t (*need_fn)(int64_t, int64_t);
  PyObject* own;
  Tensor dy, x, w, m, rs, dx, dw, db, dr, ws;
  void *h, *st;
  if (count(n, 12) || handle(a[0], &h) || matrix(a[1], "dy", &dy)) return NULL;
  const int dt = float_type(&dy, "dy");
  if (dt < 0 || matrix_like(a[2], "x", &x, dy.rows, dy.cols, dy.dtype) || vector(a[3], "weight", &w, dy.cols, 0)) return NULL;
  const int wt = float_type(&w, "weight");
  if (wt < 0 || vector(a[4], "mean", &m, dy.rows, 1) || vector(a[5], "rstd", &rs, dy.rows, 1) ||
      matrix_like(a[6], "dx", &dx, dy.rows, dy.cols, dy.dtype) || vector(a[7], "dw", &dw, dy.cols, 1) ||
      maybe_vector(a[8], "db", &db, dy.cols) || maybe(a[9], "dresidual", &dr, dy.rows, dy.cols, dy.dtype) || one_device(a + 1, 10) ||
      stream_of(a[11], a[1], &st) ||
      workspace_of(a[10], a[7], a[10] == Py_None ? ((need_fn)entry[E_LAYER_GRAD_WS])(dy.rows, dy.cols) : 0, a[11], st, &ws, &own))
    return NULL;
  const int code = ((fn)entry[E_LAYER_GRAD])(h, dy.p, x.p, w.p, m.p, rs.p, dr.p, dt, wt, dy.rows, dy.cols, dy.ld, x.ld, dr.ld, dx.p,
                                             dx.ld, dw.p, db.p, ws.p, ws.rows, st);
  give_back(own);
  return PyErr_Occurred() ? NULL : PyLong_FromLong(code);
}

/* (h, logits, ids, advantage, old_logp, ref_logp, weight, temperature, clip_low, clip_high, kl, loss, logp, dlogits, stream) */
static PyObject* policy(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, const void*, int, int64_t, int64_t, int64_t, const void*, int, const float*, const float*, const float*,
                    const float*, float, float, float, float, float*, float*, void*, int64_t, void*);
  Tensor z, ids, adv, old, ref, w, loss, logp, dz;
  void *h, *st;
  if (count(n, 15) || handle(a[0], &h) || matrix(a[1], "logits", &z)) return NULL;
  const int dt = float_type(&z, "logits");
  if (dt < 0 || vector(a[2], "ids", &ids, z.rows, 0)) return NULL;
  if (ids.dtype != dtypes[T_I32] && ids.dtype != dtypes[T_I64]) {
    PyErr_Format(PyExc_TypeError, "ids must be int32 or int64, got %S", ids.dtype);
    return NULL;
  }
  double number[4];
  for (int i = 0; i < 4; ++i) number[i] = PyFloat_AsDouble(a[7 + i]);
  if (PyErr_Occurred() || maybe_vector(a[3], "advantage", &adv, z.rows) || maybe_vector(a[4], "old_logp", &old, z.rows) ||
      maybe_vector(a[5], "ref_logp", &ref, z.rows) || maybe_vector(a[6], "weight", &w, z.rows) ||
      maybe_vector(a[11], "loss", &loss, z.rows) || maybe_vector(a[12], "logp", &logp, z.rows) ||
      maybe(a[13], "dlogits", &dz, z.rows, z.cols, z.dtype))
    return NULL;
  PyObject* tensors[9] = {a[1], a[2], a[3], a[4], a[5], a[6], a[11], a[12], a[13]};
  if (one_device(tensors, 9) || stream_of(a[14], a[1], &st)) return NULL;
  return PyLong_FromLong(((fn)entry[E_POLICY])(h, z.p, dt, z.rows, z.cols, z.ld, ids.p, ids.dtype == dtypes[T_I32] ? 32 : 64, adv.p, old.p,
                                               ref.p, w.p, (float)number[0], (float)number[1], (float)number[2], (float)number[3], loss.p,
                                               logp.p, dz.p, dz.ld, st));
}

/* (tensors, a tuple) -> (code, the library's list in a capsule or None, its calls' workspace bytes) */
#define LIST_NAME "precond_list"
static void list_end(PyObject* capsule) {
  typedef int (*fn)(void*);
  ((fn)entry[E_LIST_END])(PyCapsule_GetPointer(capsule, LIST_NAME));
}
static PyObject* tensor_list(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void**, int, void* const*, const int*, const int64_t*);
  typedef int64_t (*need_fn)(void*);
  if (count(n, 1)) return NULL;
  if (!PyTuple_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "tensors must be a tuple");
    return NULL;
  }
  const Py_ssize_t many = PyTuple_GET_SIZE(a[0]);
  if (many > 1 << 24) {
    PyErr_SetString(PyExc_ValueError, "too many tensors");
    return NULL;
  }
  PyObject *out = NULL, *capsule = NULL;
  void** p = PyMem_Malloc((many + 1) * sizeof(void*));
  int* types = PyMem_Malloc((many + 1) * sizeof(int));
  int64_t* sizes = PyMem_Malloc((many + 1) * sizeof(int64_t));
  void* list = NULL;
  if (!p || !types || !sizes) {
    PyErr_NoMemory();
    goto done;
  }
  for (Py_ssize_t i = 0; i < many; ++i) {
    Tensor t;
    if (get_as(PyTuple_GET_ITEM(a[0], i), "a tensor of the list", &t, 1)) goto done;
    if (!t.dense) {
      PyErr_Format(PyExc_ValueError, "tensor %zd of the list has gaps between its elements", i);
      goto done;
    }
    if ((types[i] = float_type(&t, "a tensor of the list")) < 0) goto done;
    p[i] = t.p;
    sizes[i] = t.rows;
  }
  if (many && one_device(&PyTuple_GET_ITEM(a[0], 0), many)) goto done;
  const int code = ((fn)entry[E_LIST])(&list, (int)many, p, types, sizes);
  if (code == 0 && !(capsule = PyCapsule_New(list, LIST_NAME, list_end))) goto done;
  out = capsule ? Py_BuildValue("(iNL)", code, capsule, (long long)((need_fn)entry[E_LIST_WS])(list)) : Py_BuildValue("(iOL)", code, Py_None, 0ll);
done:
  PyMem_Free(p);
  PyMem_Free(types);
  PyMem_Free(sizes);
  return out;
}

/* (h, list, first tensor or None, norm, workspace, stream) and (h, list, first tensor or None, max_norm, norm, given,
 * workspace, stream) */
static int list_call(PyObject* list, PyObject* first, PyObject* norm, PyObject* workspace, PyObject* stream, int given, void** l, Tensor* o,
                     void** st, Tensor* ws, PyObject** own) {
  typedef int64_t (*need_fn)(void*);
  *own = NULL;
  if (!(*l = PyCapsule_GetPointer(list, LIST_NAME)) || get(norm, "norm", o)) return -1;
  if (o->rows * o->cols != 1 || o->dtype != dtypes[T_F32]) return bad(PyExc_ValueError, "norm", "must be one torch.float32 number");
  PyObject* tensors[3] = {norm, first, workspace};
  if (one_device(tensors, 3) || stream_of(stream, norm, st)) return -1;
  return workspace_of(workspace, norm, workspace == Py_None && !given ? ((need_fn)entry[E_LIST_WS])(*l) : 0, stream, *st, ws, own);
}
static PyObject* grad_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, void*, float*, void*, int64_t, void*);
  PyObject* own;
  Tensor norm, ws;
  void *h, *st, *l;
  if (count(n, 6) || handle(a[0], &h) || list_call(a[1], a[2], a[3], a[4], a[5], 0, &l, &norm, &st, &ws, &own)) return NULL;
  const int code = ((fn)entry[E_GRAD_NORM])(h, l, norm.p, ws.p, ws.rows, st);
  give_back(own);
  return PyErr_Occurred() ? NULL : PyLong_FromLong(code);
}
static PyObject* clip_grads(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  typedef int (*fn)(void*, void*, float, float*, int, void*, int64_t, void*);
  PyObject* own;
  Tensor norm, ws;
  void *h, *st, *l;
  if (count(n, 8) || handle(a[0], &h)) return NULL;
  const double most = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) return NULL;
  const int given = PyObject_IsTrue(a[5]);
  if (given < 0 || list_call(a[1], a[2], a[4], a[6], a[7], given, &l, &norm, &st, &ws, &own)) return NULL;
  const int code = ((fn)entry[E_CLIP])(h, l, (float)most, norm.p, given, ws.p, ws.rows, st);
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
    {"layer_norm", (PyCFunction)(void (*)(void))layer_norm, METH_FASTCALL, NULL},
    {"layer_norm_grad", (PyCFunction)(void (*)(void))layer_norm_grad, METH_FASTCALL, NULL},
    {"policy", (PyCFunction)(void (*)(void))policy, METH_FASTCALL, NULL},
    {"tensor_list", (PyCFunction)(void (*)(void))tensor_list, METH_FASTCALL, NULL},
    {"grad_norm", (PyCFunction)(void (*)(void))grad_norm, METH_FASTCALL, NULL},
    {"clip_grads", (PyCFunction)(void (*)(void))clip_grads, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods};

PyMODINIT_FUNC PyInit__binding(void) {
  if (!(s_shape = PyUnicode_InternFromString("shape")) || !(s_stride = PyUnicode_InternFromString("stride")) ||
      !(s_is_contiguous = PyUnicode_InternFromString("is_contiguous")) ||
      !(s_data_ptr = PyUnicode_InternFromString("data_ptr")) || !(s_dtype = PyUnicode_InternFromString("dtype")) ||
      !(s_get_device = PyUnicode_InternFromString("get_device")) || !(s_new_empty = PyUnicode_InternFromString("new_empty")))
    return NULL;
  return PyModule_Create(&module);
}
