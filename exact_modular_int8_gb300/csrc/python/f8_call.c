/*
 * f8_call.c -- the Python binding's short way into quantize_f8, scaled_gemm_f8
 * and linear_f8 with its backward pass (include/resgemm.h).
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
typedef int (*capturing_fn)(void*);

static quantize_fn lib_quantize;
static gemm_fn lib_gemm;
static linear_fn lib_linear;
static backward_fn lib_backward;
static bytes_fn lib_saved_bytes, lib_ws_bytes;
static capturing_fn lib_capturing;
static PyObject *types[3], *f8_type, *byte_type; /* torch dtypes by RG_TYPE_*, E4M3, uint8 */
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
/* The two entries of a tuple; 0 if it is not a pair of integers. */
static int two(PyObject* t, int64_t* a, int64_t* b) {
  int ok = 0;
  if (t && PyTuple_Check(t) && PyTuple_GET_SIZE(t) == 2) {
    *a = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 0));
    *b = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 1));
    ok = !PyErr_Occurred();
  }
  Py_XDECREF(t);
  return ok;
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
static void* data_of(PyObject* t) { return (void*)(uintptr_t)call_int(t, s_data_ptr); }

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

/* backward(dY, saved, M, N, K, dw_dtype, flags) -> (dX, dW); None to decline */
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
  PyObject* dX = new_matrix(M, K, types[t], device);
  PyObject* dW = dX ? new_matrix(N, K, types[tw], device) : NULL;
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

/* setup((seven addresses), (f32, f16, bf16), f8, uint8, empty, empty_strided, raw_stream, current_device, workspaces,
 * raise) */
static PyObject* setup(PyObject* self, PyObject* args) {
  (void)self;
  unsigned long long f[7];
  PyObject *t0, *t1, *t2;
  if (!PyArg_ParseTuple(args, "(KKKKKKK)(OOO)OOOOOOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &t0, &t1, &t2,
                        &f8_type, &byte_type, &empty, &empty_strided, &raw_stream, &current_device, &workspaces,
                        &raise_status))
    return NULL;
  lib_quantize = (quantize_fn)(uintptr_t)f[0];
  lib_gemm = (gemm_fn)(uintptr_t)f[1];
  lib_linear = (linear_fn)(uintptr_t)f[2];
  lib_backward = (backward_fn)(uintptr_t)f[3];
  lib_saved_bytes = (bytes_fn)(uintptr_t)f[4];
  lib_ws_bytes = (bytes_fn)(uintptr_t)f[5];
  lib_capturing = (capturing_fn)(uintptr_t)f[6];
  types[RG_TYPE_F32] = t0;
  types[RG_TYPE_F16] = t1;
  types[RG_TYPE_BF16] = t2;
  PyObject* keep[] = {t0,         t1,         t2,         f8_type,        byte_type,  empty, empty_strided,
                      raw_stream, current_device, workspaces, raise_status};
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
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "f8_call", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit_f8_call(void) { return PyModule_Create(&module); }
