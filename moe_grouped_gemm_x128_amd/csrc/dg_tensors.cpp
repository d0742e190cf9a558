// dg_tensors.cpp -- the binding's checks of a tensor: type, shape, GPU and
// layout in one step, and its address (Python module _tensors).
//
// Small calls are bound by what happens before the launch: asked through
// Python, the five questions about one tensor take 0.45 us, and a call has five
// to ten tensors.  The answers and the refusals are the same as in Python: where
// anything does not match, the functions that refuse_with() and otherwise() were
// given are called with the same arguments, and raise.  The binding does the same in
// Python alone where this module is missing or was built with another torch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <float.h>
#include <limits.h>
#include <math.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dg.h"

namespace {

PyObject* g_refuse = nullptr;

PyObject* refuse(PyObject* const* args) {
  if (!g_refuse) {
    PyErr_SetString(PyExc_RuntimeError, "refuse_with() was not called");
    return nullptr;
  }
  PyObject* r = PyObject_CallFunctionObjArgs(g_refuse, args[0], args[1], args[2], args[3], args[4], nullptr);
  if (r) {  // (it always raises)
    Py_DECREF(r);
    PyErr_SetString(PyExc_ValueError, "tensor refused");
  }
  return nullptr;
}

// Whether args = (tensor, dtype, shape, device index, name) match.  Null and an
// error set if they are not of those types.
const at::Tensor* matched(PyObject* const* args, Py_ssize_t n, bool* fits) {
  *fits = false;
  if (n != 5 || !THPDtype_Check(args[1]) || !PyTuple_Check(args[2]) || !PyLong_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "expected (tensor, dtype, shape, device index, name)");
    return nullptr;
  }
  if (!THPVariable_Check(args[0])) {
    PyErr_Format(PyExc_TypeError, "%S must be a tensor, got %R", args[4], (PyObject*)Py_TYPE(args[0]));
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(args[0]);
  const Py_ssize_t dims = PyTuple_GET_SIZE(args[2]);
  const long dev = PyLong_AsLong(args[3]);
  if (dev == -1 && PyErr_Occurred()) return nullptr;
  if (t.layout() != at::kStrided || t.scalar_type() != reinterpret_cast<THPDtype*>(args[1])->scalar_type ||
      t.dim() != dims || t.device().index() != dev || !t.is_cuda())
    return &t;
  for (Py_ssize_t i = 0; i < dims; ++i) {
    const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(args[2], i));
    if (want == -1 && PyErr_Occurred()) return nullptr;
    if (t.size(i) != want) return &t;
  }
  *fits = true;
  return &t;
}

PyObject* address(const at::Tensor& t) { return PyLong_FromVoidPtr(t.data_ptr()); }

PyObject* whole(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool fits;
  const at::Tensor* t = matched(args, n, &fits);
  if (!t) return nullptr;
  if (!fits || !t->is_contiguous()) return refuse(args);
  return address(*t);
  END_HANDLE_TH_ERRORS
}

PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool fits;
  const at::Tensor* t = matched(args, n, &fits);
  if (!t) return nullptr;
  if (!fits || t->dim() != 2) return refuse(args);
  const int64_t m = t->size(0), cols = t->size(1);
  const int64_t ld = t->stride(0), one = t->stride(1);
  if ((one != 1 && cols > 1) || (ld < cols && m > 1)) return refuse(args);
  PyObject* at = address(*t);
  if (!at) return nullptr;
  // (one row: its stride may be anything)
  PyObject* stride = PyLong_FromLongLong(m > 1 ? ld : cols);
  PyObject* both = stride ? PyTuple_Pack(2, at, stride) : nullptr;
  Py_DECREF(at);
  Py_XDECREF(stride);
  return both;
  END_HANDLE_TH_ERRORS
}

// ---- whole arguments of a call: on any mismatch the Python function of the
// same name answers ----
enum Which { kMatrix, kVector, kBytes8, kLayout, kSlots, kNorm, kCount };
PyObject* g_otherwise[kCount] = {};

PyObject* otherwise(Which w, PyObject* const* args, Py_ssize_t n) {
  if (!g_otherwise[w]) {
    PyErr_SetString(PyExc_RuntimeError, "otherwise() was not called");
    return nullptr;
  }
  PyErr_Clear();  // (of a number that did not convert: the function says what is wrong)
  return PyObject_Vectorcall(g_otherwise[w], args, n, nullptr);
}

// The tensor `o` if it is a strided one on GPU `dev` (dev < 0: on any).
const at::Tensor* tensor_on(PyObject* o, long dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == at::kStrided && t.is_cuda() && (dev < 0 || t.device().index() == dev) ? &t : nullptr;
}

long device_of(PyObject* o) {  // (a number that is none: no tensor is on it)
  const long dev = PyLong_Check(o) ? PyLong_AsLong(o) : LONG_MAX;
  return dev < 0 ? LONG_MAX : dev;
}

PyObject* address_and(const at::Tensor& t, int64_t n) {
  PyObject* at = address(t);
  PyObject* number = at ? PyLong_FromLongLong(n) : nullptr;
  PyObject* both = number ? PyTuple_Pack(2, at, number) : nullptr;
  Py_XDECREF(at);
  Py_XDECREF(number);
  return both;
}

int vector_kind(const at::Tensor& t) {  // dg_type, -1: none
  return t.scalar_type() == at::kBFloat16 ? 0 : t.scalar_type() == at::kFloat ? 1 : -1;
}
bool is_bytes8(const at::Tensor& t) { return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn; }

// (t, name, function that gives the current GPU) -> shape, GPU
PyObject* matrix(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* t = n == 3 ? tensor_on(args[0], -1) : nullptr;
  if (!t || t->dim() != 2) return otherwise(kMatrix, args, n);
  PyObject* current = PyObject_CallNoArgs(args[2]);
  if (!current) return nullptr;
  if (device_of(current) != t->device().index()) {
    Py_DECREF(current);
    return otherwise(kMatrix, args, n);
  }
  return Py_BuildValue("((LL)N)", (long long)t->size(0), (long long)t->size(1), current);
  END_HANDLE_TH_ERRORS
}

// (t, n, GPU, name) -> address, dg_type
PyObject* vector(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* t = n == 4 ? tensor_on(args[0], device_of(args[2])) : nullptr;
  if (!t || t->dim() != 1 || vector_kind(*t) < 0 || !t->is_contiguous() || !PyLong_Check(args[1]) ||
      PyLong_AsLongLong(args[1]) != t->size(0))
    return otherwise(kVector, args, n);
  return address_and(*t, vector_kind(*t));
  END_HANDLE_TH_ERRORS
}

// (t, shape, GPU, name) -> address
PyObject* bytes8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* t = n == 4 ? tensor_on(args[0], device_of(args[2])) : nullptr;
  if (!t || t->dim() != 2 || !is_bytes8(*t) || !t->is_contiguous() || !PyTuple_Check(args[1]) ||
      PyTuple_GET_SIZE(args[1]) != 2 || PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], 0)) != t->size(0) ||
      PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], 1)) != t->size(1))
    return otherwise(kBytes8, args, n);
  return address(*t);
  END_HANDLE_TH_ERRORS
}

// (a, dtype or None, columns, GPU, name) -> address, rows
PyObject* layout(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* t = n == 5 ? tensor_on(args[0], device_of(args[3])) : nullptr;
  if (!t || (t->dim() != 2 && t->dim() != 3) || !t->is_contiguous() || !PyLong_Check(args[2]) ||
      PyLong_AsLongLong(args[2]) != t->size(t->dim() - 1) ||
      !(args[1] == Py_None ? is_bytes8(*t)
                           : THPDtype_Check(args[1]) && reinterpret_cast<THPDtype*>(args[1])->scalar_type == t->scalar_type()))
    return otherwise(kLayout, args, n);
  return address_and(*t, t->dim() == 2 ? t->size(0) : t->size(0) * t->size(1));
  END_HANDLE_TH_ERRORS
}

// (rows, tokens, GPU) -> address, top_k
PyObject* slots(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* t = n == 3 ? tensor_on(args[0], device_of(args[2])) : nullptr;
  if (!t || t->dim() != 2 || t->scalar_type() != at::kInt || !t->is_contiguous() || !PyLong_Check(args[1]) ||
      PyLong_AsLongLong(args[1]) != t->size(0))
    return otherwise(kSlots, args, n);
  return address_and(*t, t->size(1));
  END_HANDLE_TH_ERRORS
}

// (x, shape, weight, eps, residual, sum_out, rstd, GPU) -> dg_norm's bytes
// The address and row stride of bf16 rows [m, cols] (None: null); false: something else.
bool bf16_rows(PyObject* o, int64_t m, int64_t cols, long dev, const void** p, int64_t* ld) {
  if (o == Py_None) return true;
  const at::Tensor* t = tensor_on(o, dev);
  if (!t || t->dim() != 2 || t->scalar_type() != at::kBFloat16 || t->size(0) != m || t->size(1) != cols ||
      (t->stride(1) != 1 && cols > 1) || (t->stride(0) < cols && m > 1))
    return false;
  *p = t->data_ptr();
  *ld = m > 1 ? t->stride(0) : cols;
  return true;
}
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8 || args[0] == Py_None || !PyTuple_Check(args[1]) || PyTuple_GET_SIZE(args[1]) != 2 || !PyFloat_Check(args[3]))
    return otherwise(kNorm, args, n);
  const int64_t m = PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], 0)), h = PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], 1));
  const long dev = device_of(args[7]);
  dg_norm out{};
  const void* sum = nullptr;
  bool fits = m >= 0 && h >= 0 && bf16_rows(args[0], m, h, dev, &out.x, &out.ld_x) &&
              bf16_rows(args[4], m, h, dev, &out.residual, &out.ld_residual) &&
              bf16_rows(args[5], m, h, dev, &sum, &out.ld_sum) && fabs(PyFloat_AS_DOUBLE(args[3])) <= FLT_MAX;
  if (fits && args[2] != Py_None) {
    const at::Tensor* w = tensor_on(args[2], dev);
    fits = w && w->dim() == 1 && vector_kind(*w) >= 0 && w->size(0) == h && w->is_contiguous();
    if (fits) {
      out.weight = w->data_ptr();
      out.weight_type = vector_kind(*w);
    }
  }
  if (fits && args[6] != Py_None) {
    const at::Tensor* r = tensor_on(args[6], dev);
    fits = r && r->dim() == 1 && r->scalar_type() == at::kFloat && r->size(0) == m && r->is_contiguous();
    if (fits) out.rstd = static_cast<float*>(r->data_ptr());
  }
  if (!fits) return otherwise(kNorm, args, n);
  out.sum = const_cast<void*>(sum);
  out.eps = (float)PyFloat_AS_DOUBLE(args[3]);
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&out), sizeof(out));
  END_HANDLE_TH_ERRORS
}

PyObject* set_otherwise(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kCount) {
    PyErr_Format(PyExc_TypeError, "expected %d functions", (int)kCount);
    return nullptr;
  }
  for (int i = 0; i < kCount; ++i) {
    Py_INCREF(args[i]);
    Py_XSETREF(g_otherwise[i], args[i]);
  }
  Py_RETURN_NONE;
}

PyObject* refuse_with(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_refuse, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"whole", (PyCFunction)(void (*)(void))whole, METH_FASTCALL,
     "whole(tensor, dtype, shape, device, name): address of a contiguous tensor of that type and shape on that GPU"},
    {"rows", (PyCFunction)(void (*)(void))rows, METH_FASTCALL,
     "rows(tensor, dtype, shape, device, name): address and row stride of a matrix with contiguous rows"},
    {"matrix", (PyCFunction)(void (*)(void))matrix, METH_FASTCALL, "matrix(t, name, f): shape and GPU, which is f()"},
    {"vector", (PyCFunction)(void (*)(void))vector, METH_FASTCALL, "vector(t, n, GPU, name): address and dg_type"},
    {"bytes8", (PyCFunction)(void (*)(void))bytes8, METH_FASTCALL, "bytes8(t, shape, GPU, name): address"},
    {"layout", (PyCFunction)(void (*)(void))layout, METH_FASTCALL,
     "layout(a, dtype or None for FP8 bytes, columns, GPU, name): address and rows"},
    {"slots", (PyCFunction)(void (*)(void))slots, METH_FASTCALL, "slots(rows, tokens, GPU): address and top_k"},
    {"norm", (PyCFunction)(void (*)(void))norm, METH_FASTCALL,
     "norm(x, shape, weight, eps, residual, sum_out, rstd, GPU): a dg_norm as bytes"},
    {"otherwise", (PyCFunction)(void (*)(void))set_otherwise, METH_FASTCALL,
     "otherwise(matrix, vector, bytes8, layout, slots, norm): what answers where the native ones do not"},
    {"refuse_with", refuse_with, METH_O, "refuse_with(f): f(tensor, dtype, shape, device, name) raises on a mismatch"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", "The binding's checks of tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__tensors(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_with", DG_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
