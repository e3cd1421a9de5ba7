// The tensor wrappers' common case in C++: calls of operators with torch tensors whose marshalling would take
// longer in Python than the kernel's launch does.  (An RMSNorm's call with six tensors: 6.8 us in Python and
// ctypes, 4.1 by the tensors' Python attributes from C, 2.1 by the tensors themselves, of which 1.5 to 1.9 are the launch.)
//
// A function returns True when it made the call, and None when it did not: an argument is not of
// the form it takes, or the library refused the call, which changed nothing.  The caller then
// goes through the checks in Python, which say what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tqd.h"

namespace {

decltype(&tqd_op_rows_i8) op_rows;
decltype(&tqd_op_rmsnorm_i8) op_norm;
decltype(&tqd_op_silu_mul_i8) op_silu;
decltype(&tqd_op_rows_i8_read) op_read;
decltype(&tqd_op_i8_matmul) op_matmul;
decltype(&tqd_i8_matmul_scratch_bytes) matmul_scratch;
decltype(&tqd_op_rope_rows) op_rope;

// Memory that an operator takes as a pointer to whatever type it has.
struct Memory {
  void* p = nullptr;
  template <class T>
  operator T*() const {
    return static_cast<T*>(p);
  }
};

// rows and width of [rows, width], or of [width] as one row; not of classes derived from Tensor, which may mean
// something else by what they hold.
bool shape_of(PyObject* o, int64_t& n, int64_t& w) {
  if (!THPVariable_CheckExact(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  const int64_t d = t.dim();
  if (d != 1 && d != 2) return false;
  n = d == 2 ? t.size(0) : 1;
  w = t.size(d - 1);
  return n <= INT32_MAX && w <= INT32_MAX;
}

bool is_on(const at::Tensor& t, at::ScalarType dtype, int dev) {
  return t.scalar_type() == dtype && t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided;
}

// Memory and row stride of a tensor [n, w] (n 1: or [w]) of dtype on dev with contiguous rows that do not overlap.
bool rows_of(PyObject* o, at::ScalarType dtype, int dev, int64_t n, int64_t w, Memory& m, int64_t& stride) {
  int64_t tn, tw;
  if (!shape_of(o, tn, tw) || tn != n || tw != w) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!is_on(t, dtype, dev) || (w > 1 && t.stride(-1) != 1)) return false;
  stride = n > 1 ? t.stride(0) : w;
  m.p = t.data_ptr();
  return stride >= w;
}

// Memory of a contiguous tensor of at least n elements of dtype on dev.
bool vector_of(PyObject* o, at::ScalarType dtype, int dev, int64_t n, Memory& m) {
  if (!THPVariable_CheckExact(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!is_on(t, dtype, dev) || t.numel() < n || !t.is_contiguous()) return false;
  m.p = t.data_ptr();
  return true;
}

bool stream_of(PyObject* stream, int dev, void*& st) {
  if (stream == Py_None) {
    st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    return true;
  }
  PyObject* r = PyObject_GetAttrString(stream, "cuda_stream");
  if (!r) return false;
  st = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

#define CALL(made, expression)           \
  do {                                   \
    int32_t rc_;                         \
    Py_BEGIN_ALLOW_THREADS;              \
    rc_ = (expression);                  \
    Py_END_ALLOW_THREADS;                \
    made = rc_ == TQD_OK;                \
  } while (0)

bool rows_i8(PyObject* const* a, Py_ssize_t argc) {  // x, q, scale, stream
  const int dev = c10::cuda::current_device();
  bool made = false;
  int64_t n, w;
  Memory x, q, scale;
  void* st;
  int64_t xs, qs;
  if (argc == 4 && shape_of(a[0], n, w) && rows_of(a[0], at::kFloat, dev, n, w, x, xs) &&
      rows_of(a[1], at::kChar, dev, n, w, q, qs) && vector_of(a[2], at::kFloat, dev, n, scale) && stream_of(a[3], dev, st))
    CALL(made, op_rows(x, xs, static_cast<int32_t>(n), static_cast<int32_t>(w), q, qs, scale, st));
  return made;
}

bool rmsnorm_i8(PyObject* const* a, Py_ssize_t argc) {  // x, add, g, eps, sum, q, scale, stream
  const int dev = c10::cuda::current_device();
  bool made = false;
  int64_t n, w;
  Memory x, add, g, sum, q, scale;
  void* st;
  int64_t xs, as = 0, ss = 0, qs;
  if (argc == 8 && shape_of(a[0], n, w) && rows_of(a[0], at::kFloat, dev, n, w, x, xs) &&
      (a[1] == Py_None || rows_of(a[1], at::kFloat, dev, n, w, add, as)) && vector_of(a[2], at::kFloat, dev, w, g) &&
      PyFloat_Check(a[3]) && (a[4] == Py_None || rows_of(a[4], at::kFloat, dev, n, w, sum, ss)) &&
      rows_of(a[5], at::kChar, dev, n, w, q, qs) && vector_of(a[6], at::kFloat, dev, n, scale) && stream_of(a[7], dev, st)) {
    const float eps = static_cast<float>(PyFloat_AS_DOUBLE(a[3]));
    CALL(made, op_norm(x, xs, add, as, g, static_cast<int32_t>(n), static_cast<int32_t>(w), eps, sum, ss, q, qs, scale, st));
  }
  return made;
}

bool silu_mul_i8(PyObject* const* a, Py_ssize_t argc) {  // gate, up, q, scale, stream
  const int dev = c10::cuda::current_device();
  bool made = false;
  int64_t n, w;
  Memory gate, up, q, scale;
  void* st;
  int64_t gs, us, qs;
  if (argc == 5 && shape_of(a[0], n, w) && rows_of(a[0], at::kFloat, dev, n, w, gate, gs) &&
      rows_of(a[1], at::kFloat, dev, n, w, up, us) && rows_of(a[2], at::kChar, dev, n, w, q, qs) &&
      vector_of(a[3], at::kFloat, dev, n, scale) && stream_of(a[4], dev, st))
    CALL(made, op_silu(gate, gs, up, us, static_cast<int32_t>(n), static_cast<int32_t>(w), q, qs, scale, st));
  return made;
}

bool rows_i8_read(PyObject* const* a, Py_ssize_t argc) {  // q, scale, out, stream
  const int dev = c10::cuda::current_device();
  bool made = false;
  int64_t n, w;
  Memory q, scale, out;
  void* st;
  int64_t qs, os;
  if (argc == 4 && shape_of(a[0], n, w) && rows_of(a[0], at::kChar, dev, n, w, q, qs) &&
      vector_of(a[1], at::kFloat, dev, n, scale) && rows_of(a[2], at::kFloat, dev, n, w, out, os) && stream_of(a[3], dev, st))
    CALL(made, op_read(q, qs, scale, static_cast<int32_t>(n), static_cast<int32_t>(w), out, os, st));
  return made;
}

bool i8_matmul(PyObject* const* a, Py_ssize_t argc) {  // w, w_scale, x, x_scale, y, scratch, stream
  const int dev = c10::cuda::current_device();
  bool made = false;
  int64_t n, cols, rows, wc;
  Memory w, ws, x, xsc, y, scratch;
  void* st;
  int64_t xs, ys, wst;
  if (argc == 7 && shape_of(a[2], n, cols) && shape_of(a[0], rows, wc) && wc == cols &&
      rows_of(a[0], at::kChar, dev, rows, cols, w, wst) && wst == cols && vector_of(a[1], at::kFloat, dev, rows, ws) &&
      rows_of(a[2], at::kChar, dev, n, cols, x, xs) && vector_of(a[3], at::kFloat, dev, n, xsc) &&
      rows_of(a[4], at::kFloat, dev, n, rows, y, ys)) {
    const size_t need = matmul_scratch(static_cast<int32_t>(rows), static_cast<int32_t>(cols), static_cast<int32_t>(n));
    if ((!need || (a[5] != Py_None && vector_of(a[5], at::kByte, dev, static_cast<int64_t>(need), scratch))) && stream_of(a[6], dev, st))
      CALL(made, op_matmul(w, ws, static_cast<int32_t>(rows), static_cast<int32_t>(cols), x, xs, xsc, static_cast<int32_t>(n), y, ys,
                           scratch, st));
  }
  return made;
}

bool rope_rows(PyObject* const* a, Py_ssize_t argc) {
  // x, positions, table, head_dim, rotary_dim, interleaved, out, stream
  const int dev = c10::cuda::current_device();
  bool made = false;
  int64_t n, w;
  Memory x, pos, table, out;
  void* st;
  int64_t xs, os;
  if (argc == 8 && PyLong_Check(a[3]) && PyLong_Check(a[4]) && shape_of(a[0], n, w)) {
    const long long hd = PyLong_AsLongLong(a[3]), rot = PyLong_AsLongLong(a[4]);
    const int inter = PyObject_IsTrue(a[5]);
    if (hd > 0 && hd <= 0x7FFFFFFF && rot > 0 && rot <= hd && w % hd == 0 && inter >= 0 &&
        rows_of(a[0], at::kFloat, dev, n, w, x, xs) && vector_of(a[1], at::kInt, dev, n, pos) && vector_of(a[2], at::kFloat, dev, rot, table) &&
        rows_of(a[6], at::kFloat, dev, n, w, out, os) && stream_of(a[7], dev, st)) {
      const int64_t entries = THPVariable_Unpack(a[2]).numel();
      if (entries % rot == 0 && entries / rot <= 0x7FFFFFFF)
        CALL(made, op_rope(x, xs, pos, static_cast<int32_t>(n), static_cast<int32_t>(w / hd), static_cast<int32_t>(hd), table,
                           static_cast<int32_t>(entries / rot), static_cast<int32_t>(rot), inter, out, os, st));
    }
  }
  return made;
}

template <bool (*kCall)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t argc) {
  bool made = false;
  try {
    made = kCall(a, argc);
  } catch (...) {  // (a tensor without memory, no device)
  }
  PyErr_Clear();
  if (made) Py_RETURN_TRUE;
  Py_RETURN_NONE;
}

template <class F>
bool find(void* lib, const char* name, F& f) {
  f = reinterpret_cast<F>(dlsym(lib, name));
  return f != nullptr;
}

// bind(library path): before any other call.
PyObject* bind(PyObject*, PyObject* args) {
  const char* path;
  if (!PyArg_ParseTuple(args, "s", &path)) return nullptr;
  void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return nullptr;
  }
  if (!find(lib, "tqd_op_rows_i8", op_rows) || !find(lib, "tqd_op_rmsnorm_i8", op_norm) ||
      !find(lib, "tqd_op_silu_mul_i8", op_silu) || !find(lib, "tqd_op_rows_i8_read", op_read) ||
      !find(lib, "tqd_op_i8_matmul", op_matmul) || !find(lib, "tqd_i8_matmul_scratch_bytes", matmul_scratch) ||
      !find(lib, "tqd_op_rope_rows", op_rope)) {
    PyErr_SetString(PyExc_ImportError, "an operator is missing from the library");
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rows_i8),   FAST(rmsnorm_i8), FAST(silu_mul_i8), FAST(rows_i8_read),
                         FAST(i8_matmul), FAST(rope_rows),  {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tqd_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tqd_call() { return PyModule_Create(&module); }
