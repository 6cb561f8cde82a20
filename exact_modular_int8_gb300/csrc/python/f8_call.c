/*
 * f8_call.c -- the Python binding's short way into the 8-bit operators
 * (include/resgemm.h): quantisation, products, linear layers with their backward
 * passes.
 *
 * A small call's time is its time on the host, and much of that was spent on
 * marshalling: 5 of a product's or a quantisation's 13 us in the interpreter and
 * ctypes, 4 of the 16 that each pass of a linear layer took.  These functions take the tensors
 * of an ordinary call -- the current device's, rows contiguous and aligned,
 * shapes that agree -- allocate the results and call the library.  For
 * anything else they return None, and the caller's Python code checks, copies
 * or refuses the arguments as it does without them.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../../include/resgemm.h"

typedef int (*quantize_fn)(const void*, int, int64_t, int64_t, int64_t, int, uint8_t*, int64_t, float*, uint8_t*,
                           int64_t, float*, unsigned, void*);
typedef int (*gemm_fn)(const uint8_t*, int64_t, const float*, const uint8_t*, int64_t, const float*, void*, int,
                       int64_t, int64_t, int64_t, int64_t, unsigned, void*, size_t, void*);

typedef int (*linear_fn)(const void*, int, int64_t, const void*, int, int64_t, void*, int64_t, int64_t, int64_t, void*,
                         size_t, unsigned, void*, size_t, void*);
typedef int (*backward_fn)(const void*, int, int64_t, const void*, size_t, void*, void*, int, int64_t, int64_t, int64_t,
                           unsigned, void*, size_t, void*);
typedef size_t (*bytes_fn)(int64_t, int64_t, int64_t);
typedef int (*act_fn)(const void*, int64_t, const float*, const uint8_t*, int64_t, const float*, const void*, int, int,
                      const void*, int64_t, void*, void*, int, int64_t, int64_t, int64_t, int64_t, unsigned, void*, size_t,
                      void*);
typedef int (*linear_act_fn)(const void*, int, int64_t, const void*, int, int64_t, const void*, int, int, const void*,
                             int64_t, void*, int64_t, int64_t, int64_t, void*, size_t, unsigned, void*, size_t, void*);
typedef int (*linear_act_backward_fn)(const void*, int, int64_t, const void*, size_t, int, void*, void*, int, void*, int,
                                      int64_t, int64_t, int64_t, unsigned, void*, size_t, void*);
typedef size_t (*act_bytes_fn)(int64_t, int64_t, int64_t, int, int);
typedef int (*rows_fn)(const uint8_t*, int64_t, const float*, const uint8_t*, int64_t, const float*, const void*, int64_t,
                       void*, int, int64_t, int64_t, int64_t, int64_t, unsigned, void*, size_t, void*);
typedef int (*sums_fn)(const uint8_t*, int64_t, const float*, const uint8_t*, int64_t, const float*, const void*, int64_t,
                       void*, int, int64_t, int64_t, int64_t, unsigned, void*, size_t, void*);
typedef int (*expert_fn)(const void*, int, int64_t, const void*, int, int64_t, const void*, int64_t, void*, int64_t,
                         int64_t, int64_t, void*, size_t, unsigned, void*, size_t, void*);
typedef int (*expert_backward_fn)(const void*, int, int64_t, const void*, size_t, const void*, int64_t, void*, void*, int,
                                  int64_t, int64_t, int64_t, unsigned, void*, size_t, void*);
typedef int (*quantize_grouped_fn)(const void*, int, int64_t, int64_t, int64_t, int, const void*, int64_t, uint8_t*,
                                   int64_t, float*, uint8_t*, int64_t, float*, unsigned, void*);
typedef size_t (*expert_bytes_fn)(int64_t, int64_t, int64_t, int64_t);
typedef int (*capturing_fn)(void*);

static quantize_fn lib_quantize;
static gemm_fn lib_gemm;
static linear_fn lib_linear;
static backward_fn lib_backward;
static bytes_fn lib_saved_bytes, lib_ws_bytes, lib_act_ws_bytes;
static act_fn lib_act;
static linear_act_fn lib_linear_act;
static linear_act_backward_fn lib_linear_act_backward;
static act_bytes_fn lib_act_saved_bytes;
static rows_fn lib_rows;
static sums_fn lib_sums;
static expert_fn lib_expert;
static expert_backward_fn lib_expert_backward;
static quantize_grouped_fn lib_quantize_grouped;
static expert_bytes_fn lib_expert_saved_bytes, lib_expert_ws_bytes;
static capturing_fn lib_capturing;
static PyObject *types[3], *f8_type, *byte_type; /* torch dtypes by RG_TYPE_*, E4M3, uint8 */
static PyObject *int_type, *long_type;           /* of offsets */
static PyObject *empty, *empty_strided, *raw_stream, *current_device; /* torch functions */
static PyObject *workspaces, *raise_status;  /* the binding's workspace cache and error function */
static PyObject *s_shape, *s_stride, *s_dtype, *s_device, *s_data_ptr, *s_get_device, *s_numel, *empty_names;

static int64_t blocks(int64_t x) { return (x + 127) / 128; }
static int64_t up16(int64_t x) { return (x + 15) & ~(int64_t)15; }

/* A method's or function's integer result; -1 with an exception set on failure. */
static int64_t as_int(PyObject* r) {
  if (!r) return -1;
  const int64_t v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return v;
}
static int64_t call_int(PyObject* o, PyObject* name) { return as_int(PyObject_CallMethodNoArgs(o, name)); }

static PyObject* pair_of(int64_t a, int64_t b) {
  PyObject *t = PyTuple_New(2), *x = PyLong_FromLongLong(a), *y = PyLong_FromLongLong(b);
  if (t && x && y) {
    PyTuple_SET_ITEM(t, 0, x);
    PyTuple_SET_ITEM(t, 1, y);
    return t;
  }
  Py_XDECREF(t);
  Py_XDECREF(x);
  Py_XDECREF(y);
  return NULL;
}
/* The n entries of a tuple (stolen); 0 if it is not one of n integers. */
static int entries(PyObject* t, Py_ssize_t n, int64_t* v) {
  int ok = t && PyTuple_Check(t) && PyTuple_GET_SIZE(t) == n;
  for (Py_ssize_t i = 0; ok && i < n; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    ok = !(v[i] == -1 && PyErr_Occurred());
  }
  Py_XDECREF(t);
  return ok;
}
static int two(PyObject* t, int64_t* a, int64_t* b) {
  int64_t v[2];
  if (!entries(t, 2, v)) return 0;
  *a = v[0];
  *b = v[1];
  return 1;
}

typedef struct {
  int64_t m, k, ld;
  void* p;
} matrix;

/* The RG_TYPE_* of a tensor's dtype, or 3; E4M3 is 4. */
static int type_of(PyObject* t) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return 3;
  Py_DECREF(d); /* dtypes live for good */
  int i = 0;
  while (i < 3 && types[i] != d) ++i;
  return d == f8_type ? 4 : i;
}
/* A matrix with contiguous rows on device `dev` (-1: known to be there); 0 to decline. */
static int matrix_of(PyObject* t, int64_t dev, matrix* x) {
  int64_t s0, s1;
  if (dev >= 0 && call_int(t, s_get_device) != dev) return 0;
  if (!two(PyObject_GetAttr(t, s_shape), &x->m, &x->k) || !two(PyObject_CallMethodNoArgs(t, s_stride), &s0, &s1))
    return 0;
  if (x->k > 1 && s1 != 1) return 0;
  x->ld = x->m > 1 ? s0 : x->k;
  if (x->ld < x->k || !x->k || !x->m) return 0;
  x->p = (void*)(uintptr_t)call_int(t, s_data_ptr);
  return x->p && !PyErr_Occurred();
}
/* fp32 scales; 0 to decline */
static int scales_of(PyObject* t, int64_t dev, matrix* x) {
  return type_of(t) == RG_TYPE_F32 && matrix_of(t, dev, x) && x->ld == x->k;
}
/* E4M3 rows on 16-byte boundaries. */
static int values_of(PyObject* t, int64_t dev, matrix* x) {
  if (type_of(t) != 4 || !matrix_of(t, dev, x)) return 0;
  if (x->m == 1) x->ld = up16(x->ld);
  return !(x->ld & 15) && !((uintptr_t)x->p & 15);
}

/* A floating-point matrix with contiguous rows, and its RG_TYPE_*; -1 to decline. */
static int real_of(PyObject* t, int64_t dev, matrix* x) {
  const int i = type_of(t);
  return i < 3 && matrix_of(t, dev, x) ? i : -1;
}

/* A stack of matrices [e][m][k] with contiguous rows and no gaps; 0 to decline. */
typedef struct {
  int64_t e, m, k, ld;
  void* p;
} stack;
static int stack_of(PyObject* t, int64_t dev, stack* x) {
  int64_t n[3], s[3];
  if (call_int(t, s_get_device) != dev || !entries(PyObject_GetAttr(t, s_shape), 3, n) ||
      !entries(PyObject_CallMethodNoArgs(t, s_stride), 3, s))
    return 0;
  x->e = n[0];
  x->m = n[1];
  x->k = n[2];
  x->ld = s[1];
  if (!x->e || x->m < 2 || x->k < 2 || s[2] != 1 || x->ld < x->k || (x->e > 1 && s[0] != x->m * x->ld)) return 0;
  x->p = (void*)(uintptr_t)call_int(t, s_data_ptr);
  return x->p && !PyErr_Occurred();
}
/* fp32 scales of a stack */
static int stack_scales_of(PyObject* t, int64_t dev, int64_t e, int64_t m, int64_t k, void** p) {
  int64_t n[3], s[3];
  if (type_of(t) != RG_TYPE_F32 || call_int(t, s_get_device) != dev || !entries(PyObject_GetAttr(t, s_shape), 3, n) ||
      !entries(PyObject_CallMethodNoArgs(t, s_stride), 3, s))
    return 0;
  if (n[0] != e || n[1] != m || n[2] != k || s[2] != 1 || s[1] != k || s[0] != m * k) return 0;
  *p = (void*)(uintptr_t)call_int(t, s_data_ptr);
  return *p && !PyErr_Occurred();
}
/* A contiguous vector of n entries (any number for n < 0). */
static int vector_of(PyObject* t, int64_t dev, int64_t* n, void** p) {
  int64_t size, step;
  if (call_int(t, s_get_device) != dev || !entries(PyObject_GetAttr(t, s_shape), 1, &size) ||
      !entries(PyObject_CallMethodNoArgs(t, s_stride), 1, &step) || step != 1 || (*n >= 0 && size != *n))
    return 0;
  *n = size;
  *p = (void*)(uintptr_t)call_int(t, s_data_ptr);
  return *p && !PyErr_Occurred();
}
/* Offsets of e groups (any number for e < 0) and their flag; 0 to decline. */
static int offsets_of(PyObject* t, int64_t dev, int64_t* e, void** p, unsigned* flags) {
  int64_t n = *e < 0 ? -1 : *e + 1;
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return 0;
  Py_DECREF(d);
  if ((d != int_type && d != long_type) || !vector_of(t, dev, &n, p) || n < 2) return 0;
  if (d == long_type) *flags |= RG_FLAG_OFFSETS64;
  *e = n - 1;
  return 1;
}

/* An uninitialised tensor of this size (stolen) on a device. */
static PyObject* new_tensor(PyObject* size, PyObject* type, PyObject* device) {
  if (!size) return NULL;
  PyObject* args[3] = {size, type, device};
  PyObject* t = PyObject_Vectorcall(empty, args, 1, empty_names);
  Py_DECREF(size);
  return t;
}
static PyObject* new_matrix(int64_t m, int64_t k, PyObject* type, PyObject* device) {
  return new_tensor(pair_of(m, k), type, device);
}
static void* data_of(PyObject* t) { return t == Py_None ? NULL : (void*)(uintptr_t)call_int(t, s_data_ptr); }
/* A gradient [m][k], or None where it is not wanted (`no`). */
static PyObject* new_gradient(unsigned no, int64_t m, int64_t k, PyObject* type, PyObject* device) {
  return no ? Py_NewRef(Py_None) : new_matrix(m, k, type, device);
}

/* The stream's cached workspace, at least `need` bytes; none under capture into a graph, whose calls have their own.
 * The tensor is held until after the call (a new reference): while the call runs without the interpreter's lock,
 * another thread may replace or drop the cached one. */
typedef struct {
  PyObject* tensor;
  void* p;
  int64_t bytes;
} workspace;
/* 0 to decline */
static int workspace_of(int64_t dev, void* stream, size_t need, workspace* w) {
  if (lib_capturing(stream)) return 0;
  PyObject* key = pair_of(dev, (int64_t)(uintptr_t)stream);
  if (!key) return 0;
  w->tensor = PyDict_GetItemWithError(workspaces, key); /* borrowed */
  Py_DECREF(key);
  if (!w->tensor) return 0;
  Py_INCREF(w->tensor);
  w->bytes = call_int(w->tensor, s_numel);
  w->p = data_of(w->tensor);
  if (!PyErr_Occurred() && w->p && (size_t)w->bytes >= need) return 1;
  Py_DECREF(w->tensor);
  return 0;
}

/* The device that holds `t`, if it is the current one, and its current stream. */
static int place(PyObject* t, int64_t* dev, void** stream) {
  *dev = call_int(t, s_get_device);
  if (*dev < 0 || as_int(PyObject_CallNoArgs(current_device)) != *dev) return 0;
  PyObject* i = PyLong_FromLongLong(*dev);
  if (!i) return 0;
  PyObject* s = PyObject_CallOneArg(raw_stream, i);
  Py_DECREF(i);
  if (!s) return 0;
  *stream = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

/* None for the caller to take the long way; errors on the way here are its to report. */
static PyObject* decline(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}
static PyObject* finish(int rc, const char* where, PyObject* result) {
  if (!rc) return result;
  Py_XDECREF(result);
  PyObject* r = PyObject_CallFunction(raise_status, "is", rc, where);
  if (r) {
    Py_DECREF(r);
    PyErr_SetString(PyExc_RuntimeError, where);
  }
  return NULL;
}

/* An E4M3 matrix with rows on 16-byte boundaries, and its scales; 0 with an exception set on failure. */
typedef struct {
  PyObject *q, *s;
  void *qp, *sp;
  int64_t ld;
} quantised;
static int new_quantised(int64_t m, int64_t k, int64_t scale_rows, PyObject* device, quantised* r) {
  r->ld = up16(k);
  r->s = NULL;
  if (r->ld == k) {
    r->q = new_matrix(m, k, f8_type, device);
  } else {
    PyObject* args[4] = {pair_of(m, k), pair_of(r->ld, 1), f8_type, device};
    r->q = args[0] && args[1] ? PyObject_Vectorcall(empty_strided, args, 2, empty_names) : NULL;
    Py_XDECREF(args[0]);
    Py_XDECREF(args[1]);
  }
  if (!r->q) return 0;
  r->qp = data_of(r->q);
  r->s = new_matrix(scale_rows, blocks(k), types[RG_TYPE_F32], device);
  if (r->s) r->sp = data_of(r->s);
  if (r->s && !PyErr_Occurred()) return 1;
  Py_CLEAR(r->q);
  Py_CLEAR(r->s);
  return 0;
}

/* quantize(X, form, flags) -> (Q, S), (QT, ST) or all four; None to decline */
static PyObject* quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 3) return decline();
  const long form = PyLong_AsLong(a[1]), flags = PyLong_AsLong(a[2]);
  int64_t dev;
  void* stream;
  matrix x;
  if (PyErr_Occurred() || !place(a[0], &dev, &stream)) return decline();
  const int t = real_of(a[0], -1, &x);
  if (t < 0) return decline();
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  quantised d = {0}, c = {0}; /* along rows (or in tiles), along columns */
  const int direct = form != RG_F8_COLUMNS, turned = form == RG_F8_COLUMNS || form == RG_F8_BOTH;
  int ok = !direct || new_quantised(x.m, x.k, form == RG_F8_TILES ? blocks(x.m) : x.m, device, &d);
  ok = ok && (!turned || new_quantised(x.k, x.m, x.k, device, &c));
  Py_DECREF(device);
  PyObject* r = NULL;
  if (ok) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = lib_quantize(x.p, t, x.ld, x.m, x.k, (int)form, d.qp, d.ld, d.sp, c.qp, c.ld, c.sp, (unsigned)flags, stream);
    Py_END_ALLOW_THREADS
    r = direct && turned ? PyTuple_Pack(4, d.q, d.s, c.q, c.s)
        : direct         ? PyTuple_Pack(2, d.q, d.s)
                         : PyTuple_Pack(2, c.q, c.s);
    if (r) r = finish(rc, "quantize_f8", r);
  }
  Py_XDECREF(d.q);
  Py_XDECREF(d.s);
  Py_XDECREF(c.q);
  Py_XDECREF(c.s);
  return r;
}

/* gemm(A, SA, B, SB, out_dtype, transb, flags) -> C; None to decline */
static PyObject* gemm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 7) return decline();
  const int transb = PyObject_IsTrue(a[5]);
  unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[6]);
  int64_t dev;
  void* stream;
  matrix A, B, SA, SB;
  if (PyErr_Occurred() || transb < 0 || !place(a[0], &dev, &stream)) return decline();
  int t = 0;
  while (t < 3 && types[t] != a[4]) ++t;
  if (t == 3 || !values_of(a[0], -1, &A) || !values_of(a[2], dev, &B)) return decline();
  const int64_t N = transb ? B.m : B.k, K = A.k, kb = blocks(K), nb = blocks(N);
  if (K != (transb ? B.k : B.m) || !scales_of(a[1], dev, &SA) || SA.m != A.m || SA.k != kb) return decline();
  if (!scales_of(a[3], dev, &SB) || (transb ? SB.k : SB.m) != kb) return decline();
  if ((transb ? SB.m : SB.k) == nb) flags |= RG_FLAG_TILE_B;
  else if ((transb ? SB.m : SB.k) != N) return decline();
  if (transb) flags |= RG_FLAG_TRANS_B;
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  workspace ws;
  if (!workspace_of(dev, stream, RG_F8_WS_BYTES, &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* C = new_matrix(A.m, N, a[4], device);
  Py_DECREF(device);
  if (!C) {
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void* c = data_of(C);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_gemm(A.p, A.ld, SA.p, B.p, B.ld, SB.p, c, t, N, A.m, N, K, flags, ws.p, (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  return finish(rc, "scaled_gemm_f8", C);
}

/* linear(X, W, flags) -> (Y, (saved, M, N, K)); None to decline */
static PyObject* linear(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 3) return decline();
  const unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[2]);
  int64_t dev;
  void* stream;
  matrix X, W;
  if (PyErr_Occurred() || !place(a[0], &dev, &stream)) return decline();
  const int tx = real_of(a[0], -1, &X), tw = tx < 0 ? -1 : real_of(a[1], dev, &W);
  if (tw < 0 || X.k != W.k) return decline();
  const int64_t M = X.m, N = W.m, K = X.k;
  const size_t kept_bytes = lib_saved_bytes(M, N, K);
  PyObject* device = kept_bytes ? PyObject_GetAttr(a[0], s_device) : NULL;
  if (!device) return decline();
  workspace ws;
  if (!workspace_of(dev, stream, lib_ws_bytes(M, N, K), &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* Y = new_matrix(M, N, types[tx], device);
  PyObject* kept = Y ? new_tensor(PyLong_FromSize_t(kept_bytes), byte_type, device) : NULL;
  Py_DECREF(device);
  if (!kept) {
    Py_XDECREF(Y);
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void *y = data_of(Y), *s = data_of(kept);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_linear(X.p, tx, X.ld, W.p, tw, W.ld, y, M, N, K, s, kept_bytes, flags, ws.p, (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  PyObject* r = Py_BuildValue("(N(NLLL))", Y, kept, (long long)M, (long long)N, (long long)K);
  return r ? finish(rc, "linear_f8", r) : NULL;
}

/* backward(dY, saved, M, N, K, dw_dtype, flags) -> (dX, dW), None for those not wanted; None to decline */
static PyObject* backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 7) return decline();
  const int64_t M = PyLong_AsLongLong(a[2]), N = PyLong_AsLongLong(a[3]), K = PyLong_AsLongLong(a[4]);
  const unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[6]);
  int64_t dev;
  void* stream;
  matrix dY;
  if (PyErr_Occurred() || !place(a[0], &dev, &stream)) return decline();
  const int t = real_of(a[0], -1, &dY);
  int tw = 0;
  while (tw < 3 && types[tw] != a[5]) ++tw;
  if (t < 0 || tw == 3 || dY.m != M || dY.k != N || K <= 0 || call_int(a[1], s_get_device) != dev) return decline();
  const int64_t kept_bytes = call_int(a[1], s_numel);
  void* s = data_of(a[1]);
  PyObject* device = PyErr_Occurred() ? NULL : PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  workspace ws;
  if (!workspace_of(dev, stream, lib_ws_bytes(M, N, K), &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* dX = new_gradient(flags & RG_FLAG_NO_DX, M, K, types[t], device);
  PyObject* dW = dX ? new_gradient(flags & RG_FLAG_NO_DW, N, K, types[tw], device) : NULL;
  Py_DECREF(device);
  if (!dW) {
    Py_XDECREF(dX);
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void *dx = data_of(dX), *dw = data_of(dW);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_backward(dY.p, t, dY.ld, s, (size_t)kept_bytes, dx, dw, tw, M, N, K, flags, ws.p, (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  PyObject* r = PyTuple_Pack(2, dX, dW);
  Py_DECREF(dX);
  Py_DECREF(dW);
  return r ? finish(rc, "linear_f8_backward", r) : NULL;
}

/* Beside a product [m][n]: a bias of n entries and a residual in type t, or None for either; 0 to decline. */
typedef struct {
  void *bias, *r;
  int type; /* of the bias */
  int64_t ldr;
} beside;
static int beside_of(PyObject* bias, PyObject* residual, int64_t dev, int64_t m, int64_t n, int t, beside* b) {
  b->bias = b->r = NULL;
  b->type = 0;
  b->ldr = n;
  if (bias != Py_None) {
    b->type = type_of(bias);
    if (b->type > 2 || !vector_of(bias, dev, &n, &b->bias)) return 0;
  }
  if (residual != Py_None) {
    matrix r;
    if (real_of(residual, dev, &r) != t || r.m != m || r.k != n) return 0;
    b->r = r.p;
    b->ldr = r.ld;
  }
  return 1;
}
static int dtype_index(PyObject* d) {
  int t = 0;
  while (t < 3 && types[t] != d) ++t;
  return t;
}

/* act(A, SA, B, SB, bias, act, residual, pre, out_dtype, flags) -> C or (C, P); None to decline */
static PyObject* act(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 10) return decline();
  const int kind = (int)PyLong_AsLong(a[5]), pre = PyObject_IsTrue(a[7]), t = dtype_index(a[8]);
  const unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[9]);
  int64_t dev;
  void* stream;
  matrix A, B, SA, SB;
  beside b;
  if (PyErr_Occurred() || t == 3 || pre < 0 || !place(a[0], &dev, &stream)) return decline();
  if (!values_of(a[0], -1, &A) || !values_of(a[2], dev, &B) || A.k != B.k) return decline();
  const int64_t kb = blocks(A.k);
  if (!scales_of(a[1], dev, &SA) || SA.m != A.m || SA.k != kb || !scales_of(a[3], dev, &SB) || SB.m != blocks(B.m) ||
      SB.k != kb || !beside_of(a[4], a[6], dev, A.m, B.m, t, &b))
    return decline();
  workspace ws;
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  if (!workspace_of(dev, stream, RG_F8_WS_BYTES, &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject *C = new_matrix(A.m, B.m, a[8], device), *P = C && pre ? new_matrix(A.m, B.m, a[8], device) : NULL;
  Py_DECREF(device);
  if (!C || (pre && !P)) {
    Py_XDECREF(C);
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void *c = data_of(C), *p = P ? data_of(P) : NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_act(A.p, A.ld, SA.p, B.p, B.ld, SB.p, b.bias, b.type, kind, b.r, b.ldr, p, c, t, B.m, A.m, B.m, A.k, flags,
               ws.p, (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  PyObject* r = P ? Py_BuildValue("(NN)", C, P) : C;
  return r ? finish(rc, "scaled_gemm_act_f8", r) : NULL;
}

/* linear_act(X, W, bias, act, residual, flags) -> (Y, saved, M, N, K); None to decline */
static PyObject* linear_act(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 6) return decline();
  const int kind = (int)PyLong_AsLong(a[3]);
  const unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[5]);
  int64_t dev;
  void* stream;
  matrix X, W;
  beside b;
  if (PyErr_Occurred() || !place(a[0], &dev, &stream)) return decline();
  const int tx = real_of(a[0], -1, &X), tw = tx < 0 ? -1 : real_of(a[1], dev, &W);
  if (tw < 0 || X.k != W.k || !beside_of(a[2], a[4], dev, X.m, W.m, tx, &b)) return decline();
  const int64_t M = X.m, N = W.m, K = X.k;
  const size_t kept_bytes = lib_act_saved_bytes(M, N, K, tx, kind);
  PyObject* device = kept_bytes ? PyObject_GetAttr(a[0], s_device) : NULL;
  if (!device) return decline();
  workspace ws;
  if (!workspace_of(dev, stream, lib_act_ws_bytes(M, N, K), &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* Y = new_matrix(M, N, types[tx], device);
  PyObject* kept = Y ? new_tensor(PyLong_FromSize_t(kept_bytes), byte_type, device) : NULL;
  Py_DECREF(device);
  if (!kept) {
    Py_XDECREF(Y);
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void *y = data_of(Y), *s = data_of(kept);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_linear_act(X.p, tx, X.ld, W.p, tw, W.ld, b.bias, b.type, kind, b.r, b.ldr, y, M, N, K, s, kept_bytes, flags,
                      ws.p, (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  PyObject* r = Py_BuildValue("(NNLLL)", Y, kept, (long long)M, (long long)N, (long long)K);
  return r ? finish(rc, "linear_act_f8", r) : NULL;
}

/* linear_act_backward(dY, saved, M, N, K, act, bias dtype or None, dw_dtype, flags) -> (dX, dW, dbias), None for those not
 * wanted; None to decline.  The caller has compared dY's dtype. */
static PyObject* linear_act_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 9) return decline();
  const int64_t M = PyLong_AsLongLong(a[2]), N = PyLong_AsLongLong(a[3]), K = PyLong_AsLongLong(a[4]);
  const int kind = (int)PyLong_AsLong(a[5]), tw = dtype_index(a[7]), tb = a[6] == Py_None ? 0 : dtype_index(a[6]);
  const unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[8]);
  int64_t dev;
  void* stream;
  matrix dY;
  if (PyErr_Occurred() || tw == 3 || tb == 3 || !place(a[0], &dev, &stream)) return decline();
  const int t = real_of(a[0], -1, &dY);
  if (t < 0 || dY.m != M || dY.k != N || K <= 0 || call_int(a[1], s_get_device) != dev) return decline();
  const int64_t kept_bytes = call_int(a[1], s_numel);
  void* s = data_of(a[1]);
  PyObject* device = PyErr_Occurred() ? NULL : PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  workspace ws;
  if (!workspace_of(dev, stream, lib_act_ws_bytes(M, N, K), &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* dX = new_gradient(flags & RG_FLAG_NO_DX, M, K, types[t], device);
  PyObject* dW = dX ? new_gradient(flags & RG_FLAG_NO_DW, N, K, types[tw], device) : NULL;
  PyObject* db = a[6] == Py_None ? Py_NewRef(Py_None) : dW ? new_tensor(PyLong_FromLongLong(N), a[6], device) : NULL;
  Py_DECREF(device);
  if (!dW || !db) {
    Py_XDECREF(dX);
    Py_XDECREF(dW);
    Py_XDECREF(db);
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void *dx = data_of(dX), *dw = data_of(dW), *dbp = data_of(db);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_linear_act_backward(dY.p, t, dY.ld, s, (size_t)kept_bytes, kind, dx, dw, tw, dbp, tb, M, N, K, flags, ws.p,
                               (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  PyObject* r = Py_BuildValue("(NNN)", dX, dW, db);
  return r ? finish(rc, "linear_act_f8_backward", r) : NULL;
}

/* rows(A, SA, B, SB, offsets, out_dtype, transb, flags) -> C; None to decline */
static PyObject* rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 8) return decline();
  const int t = dtype_index(a[5]), transb = PyObject_IsTrue(a[6]);
  unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[7]);
  int64_t dev;
  void *stream, *SB, *off;
  matrix A, SA;
  stack B;
  if (PyErr_Occurred() || t == 3 || transb < 0 || !place(a[0], &dev, &stream)) return decline();
  if (!values_of(a[0], -1, &A) || type_of(a[2]) != 4 || !stack_of(a[2], dev, &B) || (B.ld & 15) ||
      ((uintptr_t)B.p & 15))
    return decline();
  const int64_t N = transb ? B.m : B.k, K = A.k, kb = blocks(K), nb = blocks(N);
  if (K != (transb ? B.k : B.m) || !scales_of(a[1], dev, &SA) || SA.m != A.m || SA.k != kb ||
      !stack_scales_of(a[3], dev, B.e, transb ? nb : kb, transb ? kb : nb, &SB) ||
      !offsets_of(a[4], dev, &B.e, &off, &flags))
    return decline();
  if (transb) flags |= RG_FLAG_TRANS_B;
  workspace ws;
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  if (!workspace_of(dev, stream, RG_F8_WS_BYTES, &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* C = new_matrix(A.m, N, a[5], device);
  Py_DECREF(device);
  if (!C) {
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void* c = data_of(C);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_rows(A.p, A.ld, SA.p, B.p, B.ld, SB, off, B.e, c, t, N, A.m, N, K, flags, ws.p, (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  return finish(rc, "grouped_gemm_f8", C);
}

/* quantize_grouped(X, form, offsets, flags) -> (QT, ST) or (Q, S, QT, ST); None to decline */
static PyObject* quantize_grouped(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 4) return decline();
  const long form = PyLong_AsLong(a[1]);
  unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[3]);
  int64_t dev, E = -1;
  void *stream, *off;
  matrix x;
  if (PyErr_Occurred() || !place(a[0], &dev, &stream)) return decline();
  const int t = real_of(a[0], -1, &x);
  if (t < 0 || !offsets_of(a[2], dev, &E, &off, &flags)) return decline();
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  quantised d = {0}, c = {0};
  const int direct = form == RG_F8_BOTH;
  int ok = !direct || new_quantised(x.m, x.k, x.m, device, &d);
  ok = ok && new_quantised(x.k, 128 * (x.m / 128 + E), x.k, device, &c);
  Py_DECREF(device);
  PyObject* r = NULL;
  if (ok) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = lib_quantize_grouped(x.p, t, x.ld, x.m, x.k, (int)form, off, E, d.qp, d.ld, d.sp, c.qp, c.ld, c.sp, flags, stream);
    Py_END_ALLOW_THREADS
    r = direct ? PyTuple_Pack(4, d.q, d.s, c.q, c.s) : PyTuple_Pack(2, c.q, c.s);
    if (r) r = finish(rc, "quantize_f8", r);
  }
  Py_XDECREF(d.q);
  Py_XDECREF(d.s);
  Py_XDECREF(c.q);
  Py_XDECREF(c.s);
  return r;
}

/* A new stack [e][m][k]. */
static PyObject* new_stack(int64_t e, int64_t m, int64_t k, PyObject* type, PyObject* device) {
  return new_tensor(Py_BuildValue("(LLL)", (long long)e, (long long)m, (long long)k), type, device);
}

/* sums(A, SA, B, SB, offsets, out_dtype, flags) -> C; None to decline */
static PyObject* sums(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 7) return decline();
  const int t = dtype_index(a[5]);
  unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[6]);
  int64_t dev, E = -1;
  void *stream, *off;
  matrix A, B, SA, SB;
  if (PyErr_Occurred() || t == 3 || !place(a[0], &dev, &stream)) return decline();
  if (!values_of(a[0], -1, &A) || !values_of(a[2], dev, &B) || A.k != B.k || A.k % 128) return decline();
  const int64_t nb = A.k / 128;
  if (!scales_of(a[1], dev, &SA) || SA.m != A.m || SA.k != nb || !scales_of(a[3], dev, &SB) || SB.m != B.m ||
      SB.k != nb || !offsets_of(a[4], dev, &E, &off, &flags) || nb < E)
    return decline();
  workspace ws;
  PyObject* device = PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  if (!workspace_of(dev, stream, RG_F8_WS_BYTES, &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* C = new_stack(E, A.m, B.m, a[5], device);
  Py_DECREF(device);
  if (!C) {
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void* c = data_of(C);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_sums(A.p, A.ld, SA.p, B.p, B.ld, SB.p, off, E, c, t, A.m, B.m, nb, flags, ws.p, (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  return finish(rc, "grouped_wgrad_f8", C);
}

/* expert(X, W, offsets, flags) -> (Y, (saved, None, T, N, K, E)); None to decline */
static PyObject* expert(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 4) return decline();
  unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[3]);
  int64_t dev;
  void *stream, *off;
  matrix X;
  stack W;
  if (PyErr_Occurred() || !place(a[0], &dev, &stream)) return decline();
  const int tx = real_of(a[0], -1, &X), tw = type_of(a[1]);
  if (tx < 0 || tw > 2 || !stack_of(a[1], dev, &W) || X.k != W.k || !offsets_of(a[2], dev, &W.e, &off, &flags))
    return decline();
  const int64_t T = X.m, N = W.m, K = X.k, E = W.e;
  const size_t kept_bytes = lib_expert_saved_bytes(T, N, K, E);
  PyObject* device = kept_bytes ? PyObject_GetAttr(a[0], s_device) : NULL;
  if (!device) return decline();
  workspace ws;
  if (!workspace_of(dev, stream, lib_expert_ws_bytes(T, N, K, E), &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* Y = new_matrix(T, N, types[tx], device);
  PyObject* kept = Y ? new_tensor(PyLong_FromSize_t(kept_bytes), byte_type, device) : NULL;
  Py_DECREF(device);
  if (!kept) {
    Py_XDECREF(Y);
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void *y = data_of(Y), *s = data_of(kept);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_expert(X.p, tx, X.ld, W.p, tw, W.ld, off, E, y, T, N, K, s, kept_bytes, flags, ws.p, (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  PyObject* r = Py_BuildValue("(N(NOLLLL))", Y, kept, Py_None, (long long)T, (long long)N, (long long)K, (long long)E);
  return r ? finish(rc, "expert_linear_f8", r) : NULL;
}

/* expert_backward(dY, saved, offsets, T, N, K, E, dw_dtype, flags) -> (dX, dW), None for those not wanted; None to
 * decline.  offsets may be None: the copy with which `saved` begins. */
static PyObject* expert_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 9) return decline();
  const int64_t T = PyLong_AsLongLong(a[3]), N = PyLong_AsLongLong(a[4]), K = PyLong_AsLongLong(a[5]);
  int64_t E = PyLong_AsLongLong(a[6]), dev;
  const int tw = dtype_index(a[7]);
  unsigned flags = (unsigned)PyLong_AsUnsignedLong(a[8]);
  void *stream, *off;
  matrix dY;
  if (PyErr_Occurred() || tw == 3 || !place(a[0], &dev, &stream)) return decline();
  const int t = real_of(a[0], -1, &dY);
  if (t < 0 || dY.m != T || dY.k != N || E < 1 || call_int(a[1], s_get_device) != dev) return decline();
  const int64_t kept_bytes = call_int(a[1], s_numel);
  void* s = data_of(a[1]);
  if (a[2] == Py_None) {
    off = s;
    flags |= RG_FLAG_OFFSETS64;
  } else if (!offsets_of(a[2], dev, &E, &off, &flags)) {
    return decline();
  }
  const size_t need = lib_expert_ws_bytes(T, N, K, E);
  PyObject* device = PyErr_Occurred() || !need ? NULL : PyObject_GetAttr(a[0], s_device);
  if (!device) return decline();
  workspace ws;
  if (!workspace_of(dev, stream, need, &ws)) {
    Py_DECREF(device);
    return decline();
  }
  PyObject* dX = new_gradient(flags & RG_FLAG_NO_DX, T, K, types[t], device);
  PyObject* dW = !dX ? NULL : flags & RG_FLAG_NO_DW ? Py_NewRef(Py_None) : new_stack(E, N, K, types[tw], device);
  Py_DECREF(device);
  if (!dW) {
    Py_XDECREF(dX);
    Py_DECREF(ws.tensor);
    return NULL;
  }
  void *dx = data_of(dX), *dw = data_of(dW);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = lib_expert_backward(dY.p, t, dY.ld, s, (size_t)kept_bytes, off, E, dx, dw, tw, T, N, K, flags, ws.p,
                           (size_t)ws.bytes, stream);
  Py_END_ALLOW_THREADS
  Py_DECREF(ws.tensor);
  PyObject* r = Py_BuildValue("(NN)", dX, dW);
  return r ? finish(rc, "expert_linear_f8_backward", r) : NULL;
}

/* setup((nineteen addresses), (f32, f16, bf16), f8, uint8, (int32, int64), empty, empty_strided, raw_stream,
 * current_device, workspaces, raise) */
static PyObject* setup(PyObject* self, PyObject* args) {
  (void)self;
  enum { kEntries = 19 };
  uintptr_t f[kEntries];
  PyObject *t0, *t1, *t2, *addresses;
  if (!PyArg_ParseTuple(args, "O!(OOO)OO(OO)OOOOOO", &PyTuple_Type, &addresses, &t0, &t1, &t2, &f8_type, &byte_type,
                        &int_type, &long_type, &empty, &empty_strided, &raw_stream, &current_device, &workspaces,
                        &raise_status))
    return NULL;
  if (PyTuple_GET_SIZE(addresses) != kEntries) {
    PyErr_SetString(PyExc_ValueError, "setup: another number of entry points expected");
    return NULL;
  }
  for (int i = 0; i < kEntries; ++i) f[i] = (uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(addresses, i));
  if (PyErr_Occurred()) return NULL;
  lib_quantize = (quantize_fn)f[0];
  lib_gemm = (gemm_fn)f[1];
  lib_linear = (linear_fn)f[2];
  lib_backward = (backward_fn)f[3];
  lib_saved_bytes = (bytes_fn)f[4];
  lib_ws_bytes = (bytes_fn)f[5];
  lib_capturing = (capturing_fn)f[6];
  lib_act = (act_fn)f[7];
  lib_linear_act = (linear_act_fn)f[8];
  lib_linear_act_backward = (linear_act_backward_fn)f[9];
  lib_act_saved_bytes = (act_bytes_fn)f[10];
  lib_act_ws_bytes = (bytes_fn)f[11];
  lib_rows = (rows_fn)f[12];
  lib_sums = (sums_fn)f[13];
  lib_expert = (expert_fn)f[14];
  lib_expert_backward = (expert_backward_fn)f[15];
  lib_expert_saved_bytes = (expert_bytes_fn)f[16];
  lib_expert_ws_bytes = (expert_bytes_fn)f[17];
  lib_quantize_grouped = (quantize_grouped_fn)f[18];
  types[RG_TYPE_F32] = t0;
  types[RG_TYPE_F16] = t1;
  types[RG_TYPE_BF16] = t2;
  PyObject* keep[] = {t0,        t1,    t2,            f8_type,    byte_type,      int_type,
                      long_type, empty, empty_strided, raw_stream, current_device, workspaces, raise_status};
  for (size_t i = 0; i < sizeof keep / sizeof *keep; ++i) Py_INCREF(keep[i]); /* for the life of the process */
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_device = PyUnicode_InternFromString("device");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_numel = PyUnicode_InternFromString("numel");
  empty_names = Py_BuildValue("(ss)", "dtype", "device");
  if (!empty_names || !s_numel) return NULL;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, NULL},
                                {"quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL, NULL},
                                {"gemm", (PyCFunction)(void (*)(void))gemm, METH_FASTCALL, NULL},
                                {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, NULL},
                                {"backward", (PyCFunction)(void (*)(void))backward, METH_FASTCALL, NULL},
                                {"act", (PyCFunction)(void (*)(void))act, METH_FASTCALL, NULL},
                                {"linear_act", (PyCFunction)(void (*)(void))linear_act, METH_FASTCALL, NULL},
                                {"linear_act_backward", (PyCFunction)(void (*)(void))linear_act_backward, METH_FASTCALL,
                                 NULL},
                                {"quantize_grouped", (PyCFunction)(void (*)(void))quantize_grouped, METH_FASTCALL, NULL},
                                {"rows", (PyCFunction)(void (*)(void))rows, METH_FASTCALL, NULL},
                                {"sums", (PyCFunction)(void (*)(void))sums, METH_FASTCALL, NULL},
                                {"expert", (PyCFunction)(void (*)(void))expert, METH_FASTCALL, NULL},
                                {"expert_backward", (PyCFunction)(void (*)(void))expert_backward, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "f8_call", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit_f8_call(void) { return PyModule_Create(&module); }
