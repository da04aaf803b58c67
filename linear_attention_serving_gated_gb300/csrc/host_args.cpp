// host_args.cpp -- the binding's check of one tensor argument, in native code.
//
// arg(t, dtype, n, name, shape) -> device pointer of a dense CUDA tensor of one element
// type that holds at least n elements (int16 holds the bits of either 16-bit type).
// Anything else goes to the function given to otherwise(), which says what is wrong.  From
// Python the five questions take 0.35 us a tensor, and a call has six to ten; here 0.1.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* other = nullptr;

bool pointer_of(PyObject* t, PyObject* dtype, PyObject* n, void** out) {
  if (!THPVariable_Check(t) || !THPDtype_Check(dtype)) return false;
  const long long least = PyLong_AsLongLong(n);
  if (least == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  try {
    const at::Tensor& x = THPVariable_Unpack(t);
    const at::ScalarType want = reinterpret_cast<THPDtype*>(dtype)->scalar_type, have = x.scalar_type();
    const bool bits = have == at::kShort && (want == at::kHalf || want == at::kBFloat16);
    if ((have != want && !bits) || !x.is_cuda() || !x.is_contiguous() || x.numel() < least) return false;
    *out = x.data_ptr();
    return true;
  } catch (...) {  // a tensor without memory of its own
    return false;
  }
}

PyObject* arg(PyObject*, PyObject* const* args, Py_ssize_t count) {
  void* p;
  if (count == 5 && pointer_of(args[0], args[1], args[2], &p)) return PyLong_FromVoidPtr(p);
  if (!other) return PyErr_Format(PyExc_RuntimeError, "otherwise() has not been called");
  return PyObject_Vectorcall(other, args, (size_t)count, nullptr);
}

PyObject* otherwise(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(other, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"arg", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(arg)), METH_FASTCALL, nullptr},
    {"otherwise", otherwise, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host_args() { return PyModule_Create(&module); }
