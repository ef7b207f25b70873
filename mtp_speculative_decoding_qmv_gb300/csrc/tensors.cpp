// tensors.cpp -- the bindings' checks of a call's tensors, as a CPython
// extension: a decode loop calls the library every few microseconds, and a
// dozen tensors' type, device, shape and layout cost a microsecond here that
// they cost five of in Python.  Only looks: on anything unexpected it returns
// None, and the caller finds out what is wrong and raises.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// A CUDA tensor of this type on device `index`, or null.
const at::Tensor *tensor_of(PyObject *t, PyObject *dtype, long index) {
  if (!THPVariable_Check(t) || !THPDtype_Check(dtype)) return nullptr;
  const at::Tensor &x = THPVariable_Unpack(t);
  if (!x.is_cuda() || x.get_device() != index ||
      x.scalar_type() != reinterpret_cast<THPDtype *>(dtype)->scalar_type)
    return nullptr;
  return &x;
}

// fit(index, (tensor, name, dtype, shape or None), ...) -> addresses, or None
// when one is not a contiguous tensor of that type and shape on the device.
PyObject *fit(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n < 1) Py_RETURN_NONE;
  const long index = PyLong_AsLong(args[0]);
  if (index == -1 && PyErr_Occurred()) return nullptr;
  PyObject *out = PyTuple_New(n - 1);
  if (!out) return nullptr;
  for (Py_ssize_t i = 1; i < n; ++i) {
    const at::Tensor *x = nullptr;
    if (PyTuple_Check(args[i]) && PyTuple_GET_SIZE(args[i]) == 4) {
      x = tensor_of(PyTuple_GET_ITEM(args[i], 0), PyTuple_GET_ITEM(args[i], 2), index);
      PyObject *shape = PyTuple_GET_ITEM(args[i], 3);
      if (x && !x->is_contiguous()) x = nullptr;
      if (x && shape != Py_None) {
        bool same = PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == x->dim();
        for (int64_t d = 0; same && d < x->dim(); ++d)
          same = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d)) == x->size(d);
        if (PyErr_Occurred()) PyErr_Clear();
        if (!same) x = nullptr;
      }
    }
    PyObject *address = x ? PyLong_FromVoidPtr(const_cast<void *>(x->const_data_ptr())) : nullptr;
    if (!address) {
      Py_DECREF(out);
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    PyTuple_SET_ITEM(out, i - 1, address);
  }
  return out;
}

// fit_rows(index, tensor, dtype, rows, heads, dim) -> (address, elements from a
// row to the next), or None when it is not [rows, heads, dim] with contiguous
// heads.
PyObject *fit_rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 6) Py_RETURN_NONE;
  const long index = PyLong_AsLong(args[0]);
  int64_t want[3];
  for (int i = 0; i < 3; ++i) want[i] = PyLong_AsLongLong(args[3 + i]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *x = tensor_of(args[1], args[2], index);
  if (!x || x->dim() != 3) Py_RETURN_NONE;
  for (int i = 0; i < 3; ++i)
    if (x->size(i) != want[i]) Py_RETURN_NONE;
  if (x->stride(2) != 1 || (want[1] > 1 && x->stride(1) != want[2])) Py_RETURN_NONE;
  return Py_BuildValue("NL", PyLong_FromVoidPtr(const_cast<void *>(x->const_data_ptr())),
                       (long long)(want[0] > 1 ? x->stride(0) : want[1] * want[2]));
}

PyMethodDef methods[] = {
    {"fit", (PyCFunction)(void *)fit, METH_FASTCALL, "addresses of fitting tensors, or None"},
    {"fit_rows", (PyCFunction)(void *)fit_rows, METH_FASTCALL,
     "address and row stride of fitting packed rows, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
