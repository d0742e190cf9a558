// dg_tensors.cpp -- the binding's checks of a tensor: type, shape, GPU and
// layout in one step, and its address (Python module _tensors).
//
// Small calls are bound by what happens before the launch: asked through
// Python, the five questions about one tensor take 0.45 us, and a call has five
// to ten tensors.  The answers and the refusals are the same as in Python: on
// any mismatch the function that refuse_with() was given is called with the
// arguments, and raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

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
    {"refuse_with", refuse_with, METH_O, "refuse_with(f): f(tensor, dtype, shape, device, name) raises on a mismatch"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", "The binding's checks of tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__tensors(void) { return PyModule_Create(&module); }
