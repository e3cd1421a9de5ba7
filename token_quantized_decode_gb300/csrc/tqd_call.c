/* The tensor wrappers' common case in C: calls of operators with torch tensors whose
 * marshalling would take longer in Python than the kernel's launch does (an
 * RMSNorm's call with six tensors: 6.8 us in Python and ctypes, 4.1 here, of which 1.5 the launch).
 *
 * A function returns True when it made the call, and None when it did not: an argument is not of
 * the form it takes, or the library refused the call, which changed nothing. The caller then
 * goes through the checks in Python, which say what is wrong.
 *
 * Only CPython's interface is used; a tensor is asked through its attributes. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include "tqd.h"

static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_stride, *s_numel, *s_cuda_stream;
static PyObject *t_f32, *t_i32, *t_u8, *t_i8, *raw_stream, *current_device;

static __typeof__(tqd_op_rows_i8)* op_rows;
static __typeof__(tqd_op_rmsnorm_i8)* op_norm;
static __typeof__(tqd_op_silu_mul_i8)* op_silu;
static __typeof__(tqd_op_rows_i8_read)* op_read;
static __typeof__(tqd_op_i8_matmul)* op_matmul;
static __typeof__(tqd_i8_matmul_scratch_bytes)* matmul_scratch;
static __typeof__(tqd_op_rope_rows)* op_rope;

/* A whole number that a call of `name` without arguments gives; -1 with an exception where it gives none. */
static long long number(PyObject* t, PyObject* name) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return -1;
  const long long v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return v;
}

static int truth(PyObject* t, PyObject* name) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return 0;
  const int v = r == Py_True;
  Py_DECREF(r);
  return v;
}

static int is_type(PyObject* t, PyObject* dtype) {
  PyObject* r = PyObject_GetAttr(t, s_dtype);
  if (!r) return 0;
  Py_DECREF(r); /* dtypes live as long as torch does */
  return r == dtype;
}

/* rows and width of [rows, width], or of [width] as one row. */
static int shape_of(PyObject* t, Py_ssize_t* n, Py_ssize_t* w) {
  PyObject* s = PyObject_GetAttr(t, s_shape);
  int ok = 0;
  if (!s) return 0;
  if (PyTuple_Check(s)) {
    const Py_ssize_t d = PyTuple_GET_SIZE(s);
    if (d == 1 || d == 2) {
      *n = d == 2 ? PyLong_AsSsize_t(PyTuple_GET_ITEM(s, 0)) : 1;
      *w = PyLong_AsSsize_t(PyTuple_GET_ITEM(s, d - 1));
      ok = *n >= 0 && *w >= 0 && *n <= 0x7FFFFFFF && *w <= 0x7FFFFFFF;
    }
  }
  Py_DECREF(s);
  return ok;
}

/* Pointer and row stride of a tensor [n, w] (n 1: or [w]) of dtype on dev with contiguous rows that do not overlap. */
static int rows_of(PyObject* t, PyObject* dtype, int dev, Py_ssize_t n, Py_ssize_t w, void** p, int64_t* stride) {
  Py_ssize_t tn, tw;
  if (!is_type(t, dtype) || !shape_of(t, &tn, &tw) || tn != n || tw != w || number(t, s_get_device) != dev) return 0;
  *stride = w;
  if (!truth(t, s_is_contiguous)) {
    PyObject* s = PyErr_Occurred() ? NULL : PyObject_CallMethodNoArgs(t, s_stride);
    int ok = 0;
    if (s && PyTuple_Check(s) && PyTuple_GET_SIZE(s) == 2 && n > 1) {
      const Py_ssize_t a = PyLong_AsSsize_t(PyTuple_GET_ITEM(s, 0)), b = PyLong_AsSsize_t(PyTuple_GET_ITEM(s, 1));
      ok = a >= w && (b == 1 || w == 1);
      *stride = a;
    }
    Py_XDECREF(s);
    if (!ok) return 0;
  }
  *p = (void*)(uintptr_t)number(t, s_data_ptr);
  return !PyErr_Occurred();
}

/* Pointer of a contiguous tensor of at least n elements of dtype on dev. */
static int vector_of(PyObject* t, PyObject* dtype, int dev, long long n, void** p) {
  if (!is_type(t, dtype) || number(t, s_get_device) != dev || number(t, s_numel) < n || !truth(t, s_is_contiguous)) return 0;
  *p = (void*)(uintptr_t)number(t, s_data_ptr);
  return !PyErr_Occurred();
}

static int stream_of(PyObject* stream, int dev, void** st) {
  PyObject* r;
  if (stream == Py_None) {
    PyObject* d = PyLong_FromLong(dev);
    r = d ? PyObject_CallOneArg(raw_stream, d) : NULL;
    Py_XDECREF(d);
  } else {
    r = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (!r) return 0;
  *st = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

static int device_of(int* dev) {
  PyObject* r = current_device ? PyObject_CallNoArgs(current_device) : NULL;
  if (!r) return 0;
  *dev = (int)PyLong_AsLong(r);
  Py_DECREF(r);
  return *dev >= 0;
}

static PyObject* answer(int made) {
  PyErr_Clear();
  if (made) Py_RETURN_TRUE;
  Py_RETURN_NONE;
}

#define CALL(made, expression)           \
  do {                                   \
    int32_t rc_;                         \
    Py_BEGIN_ALLOW_THREADS;              \
    rc_ = (expression);                  \
    Py_END_ALLOW_THREADS;                \
    made = rc_ == TQD_OK;                \
  } while (0)

static PyObject* rows_i8(PyObject* self, PyObject* const* a, Py_ssize_t argc) { /* x, q, scale, stream */
  int dev, made = 0;
  Py_ssize_t n, w;
  void *x, *q, *scale, *st;
  int64_t xs, qs;
  (void)self;
  if (argc == 4 && device_of(&dev) && shape_of(a[0], &n, &w) && rows_of(a[0], t_f32, dev, n, w, &x, &xs) &&
      rows_of(a[1], t_i8, dev, n, w, &q, &qs) && vector_of(a[2], t_f32, dev, n, &scale) && stream_of(a[3], dev, &st))
    CALL(made, op_rows(x, xs, (int32_t)n, (int32_t)w, q, qs, scale, st));
  return answer(made);
}

static PyObject* rmsnorm_i8(PyObject* self, PyObject* const* a, Py_ssize_t argc) { /* x, add, g, eps, sum, q, scale, stream */
  int dev, made = 0;
  Py_ssize_t n, w;
  void *x, *add = NULL, *g, *sum = NULL, *q, *scale, *st;
  int64_t xs, as = 0, ss = 0, qs;
  (void)self;
  if (argc == 8 && device_of(&dev) && shape_of(a[0], &n, &w) && rows_of(a[0], t_f32, dev, n, w, &x, &xs) &&
      (a[1] == Py_None || rows_of(a[1], t_f32, dev, n, w, &add, &as)) && vector_of(a[2], t_f32, dev, w, &g) &&
      PyFloat_Check(a[3]) && (a[4] == Py_None || rows_of(a[4], t_f32, dev, n, w, &sum, &ss)) &&
      rows_of(a[5], t_i8, dev, n, w, &q, &qs) && vector_of(a[6], t_f32, dev, n, &scale) && stream_of(a[7], dev, &st)) {
    const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
    CALL(made, op_norm(x, xs, add, as, g, (int32_t)n, (int32_t)w, eps, sum, ss, q, qs, scale, st));
  }
  return answer(made);
}

static PyObject* silu_mul_i8(PyObject* self, PyObject* const* a, Py_ssize_t argc) { /* gate, up, q, scale, stream */
  int dev, made = 0;
  Py_ssize_t n, w;
  void *gate, *up, *q, *scale, *st;
  int64_t gs, us, qs;
  (void)self;
  if (argc == 5 && device_of(&dev) && shape_of(a[0], &n, &w) && rows_of(a[0], t_f32, dev, n, w, &gate, &gs) &&
      rows_of(a[1], t_f32, dev, n, w, &up, &us) && rows_of(a[2], t_i8, dev, n, w, &q, &qs) &&
      vector_of(a[3], t_f32, dev, n, &scale) && stream_of(a[4], dev, &st))
    CALL(made, op_silu(gate, gs, up, us, (int32_t)n, (int32_t)w, q, qs, scale, st));
  return answer(made);
}

static PyObject* rows_i8_read(PyObject* self, PyObject* const* a, Py_ssize_t argc) { /* q, scale, out, stream */
  int dev, made = 0;
  Py_ssize_t n, w;
  void *q, *scale, *out, *st;
  int64_t qs, os;
  (void)self;
  if (argc == 4 && device_of(&dev) && shape_of(a[0], &n, &w) && rows_of(a[0], t_i8, dev, n, w, &q, &qs) &&
      vector_of(a[1], t_f32, dev, n, &scale) && rows_of(a[2], t_f32, dev, n, w, &out, &os) && stream_of(a[3], dev, &st))
    CALL(made, op_read(q, qs, scale, (int32_t)n, (int32_t)w, out, os, st));
  return answer(made);
}

static PyObject* i8_matmul(PyObject* self, PyObject* const* a, Py_ssize_t argc) { /* w, w_scale, x, x_scale, y, scratch, stream */
  int dev, made = 0;
  Py_ssize_t n, cols, rows, wc;
  void *w, *ws, *x, *xsc, *y, *scratch = NULL, *st;
  int64_t xs, ys, wst;
  (void)self;
  if (argc == 7 && device_of(&dev) && shape_of(a[2], &n, &cols) && shape_of(a[0], &rows, &wc) && wc == cols &&
      rows_of(a[0], t_i8, dev, rows, cols, &w, &wst) && wst == cols && vector_of(a[1], t_f32, dev, rows, &ws) &&
      rows_of(a[2], t_i8, dev, n, cols, &x, &xs) && vector_of(a[3], t_f32, dev, n, &xsc) &&
      rows_of(a[4], t_f32, dev, n, rows, &y, &ys)) {
    const size_t need = matmul_scratch((int32_t)rows, (int32_t)cols, (int32_t)n);
    if ((!need || (a[5] != Py_None && vector_of(a[5], t_u8, dev, (long long)need, &scratch))) && stream_of(a[6], dev, &st))
      CALL(made, op_matmul(w, ws, (int32_t)rows, (int32_t)cols, x, xs, xsc, (int32_t)n, y, ys, scratch, st));
  }
  return answer(made);
}

static PyObject* rope_rows(PyObject* self, PyObject* const* a, Py_ssize_t argc) {
  /* x, positions, table, head_dim, rotary_dim, interleaved, out, stream */
  int dev, made = 0;
  Py_ssize_t n, w;
  void *x, *pos, *table, *out, *st;
  int64_t xs, os;
  (void)self;
  if (argc == 8 && PyLong_Check(a[3]) && PyLong_Check(a[4]) && device_of(&dev) && shape_of(a[0], &n, &w)) {
    const long long hd = PyLong_AsLongLong(a[3]), rot = PyLong_AsLongLong(a[4]);
    const int inter = PyObject_IsTrue(a[5]);
    if (hd > 0 && hd <= 0x7FFFFFFF && rot > 0 && rot <= hd && w % hd == 0 && inter >= 0 &&
        rows_of(a[0], t_f32, dev, n, w, &x, &xs) && vector_of(a[1], t_i32, dev, n, &pos) && vector_of(a[2], t_f32, dev, rot, &table) &&
        rows_of(a[6], t_f32, dev, n, w, &out, &os) && stream_of(a[7], dev, &st)) {
      const long long entries = number(a[2], s_numel);
      if (entries % rot == 0 && entries / rot <= 0x7FFFFFFF)
        CALL(made, op_rope(x, xs, pos, (int32_t)n, (int32_t)(w / hd), (int32_t)hd, table, (int32_t)(entries / rot), (int32_t)rot, inter,
                           out, os, st));
    }
  }
  return answer(made);
}

/* bind(library path, float32, int32, uint8, int8, raw stream of a device's number, current device): before any other call. */
static PyObject* bind(PyObject* self, PyObject* args) {
  const char* path;
  PyObject* t[6];
  (void)self;
  if (!PyArg_ParseTuple(args, "sOOOOOO", &path, &t[0], &t[1], &t[2], &t[3], &t[4], &t[5])) return NULL;
  void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return NULL;
  }
  op_rows = dlsym(lib, "tqd_op_rows_i8");
  op_norm = dlsym(lib, "tqd_op_rmsnorm_i8");
  op_silu = dlsym(lib, "tqd_op_silu_mul_i8");
  op_read = dlsym(lib, "tqd_op_rows_i8_read");
  op_matmul = dlsym(lib, "tqd_op_i8_matmul");
  matmul_scratch = dlsym(lib, "tqd_i8_matmul_scratch_bytes");
  op_rope = dlsym(lib, "tqd_op_rope_rows");
  if (!op_rows || !op_norm || !op_silu || !op_read || !op_matmul || !matmul_scratch || !op_rope) {
    PyErr_SetString(PyExc_ImportError, "an operator is missing from the library");
    return NULL;
  }
  for (int i = 0; i < 6; ++i) Py_INCREF(t[i]);
  t_f32 = t[0], t_i32 = t[1], t_u8 = t[2], t_i8 = t[3], raw_stream = t[4], current_device = t[5];
  Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(rows_i8),      FAST(rmsnorm_i8), FAST(silu_mul_i8), FAST(rows_i8_read),
                                FAST(i8_matmul),    FAST(rope_rows),  {"bind", bind, METH_VARARGS, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tqd_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tqd_call(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_stride = PyUnicode_InternFromString("stride");
  s_numel = PyUnicode_InternFromString("numel");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&module);
}
