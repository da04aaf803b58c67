// host_args.cpp -- the binding's checks of a tensor argument, in native code.
//
// arg(t, dtype, n, name, shape) -> device pointer of a dense tensor of the current CUDA
// device and of one element type that holds at least n elements (int16 holds the bits of either 16-bit type).
// Anything else goes to the function given to otherwise(), which says what is wrong.  From
// Python the five questions take 0.35 us a tensor, and a call has six to ten; here 0.1.
//
// rows(t, dtype, n, width) -> (device pointer, row stride) of at least n rows of at least
// `width` elements that lie together; states(t, HV, V, K) -> (device pointer, slots) of a
// dense FP32 pool [slots, HV, V, K]; place(t) -> device pointer of a tensor of the current
// device, dense or not.  They give None where t is no such thing.
#include <Python.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* other = nullptr;

bool number(PyObject* n, long long* out) {
  *out = PyLong_AsLongLong(n);
  if (*out != -1 || !PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

bool of_type(const at::Tensor& x, PyObject* dtype) {
  const at::ScalarType want = reinterpret_cast<THPDtype*>(dtype)->scalar_type, have = x.scalar_type();
  return have == want || (have == at::kShort && (want == at::kHalf || want == at::kBFloat16));
}

// Whether a tensor is in the memory of the device that the call runs on, the current one.
bool here(const at::Tensor& x) {
  if (!x.is_cuda()) return false;
  static const c10::impl::DeviceGuardImplInterface* const several = [] {  // null: there is one
    const auto* devices = c10::impl::getDeviceGuardImpl(c10::DeviceType::CUDA);
    return devices->deviceCount() > 1 ? devices : nullptr;
  }();
  return !several || x.get_device() == several->getDevice().index();
}

bool pointer_of(PyObject* t, PyObject* dtype, PyObject* n, void** out) {
  long long least;
  if (!THPVariable_Check(t) || !THPDtype_Check(dtype) || !number(n, &least)) return false;
  try {
    const at::Tensor& x = THPVariable_Unpack(t);
    if (!of_type(x, dtype) || !here(x) || !x.is_contiguous() || x.numel() < least) return false;
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

PyObject* place(PyObject*, PyObject* t) {
  if (THPVariable_Check(t)) {
    try {
      const at::Tensor& x = THPVariable_Unpack(t);
      if (here(x)) return PyLong_FromVoidPtr(x.data_ptr());
    } catch (...) {
    }
  }
  Py_RETURN_NONE;
}

PyObject* pair(void* p, long long n) {
  PyObject* pointer = PyLong_FromVoidPtr(p);
  PyObject* value = PyLong_FromLongLong(n);
  PyObject* both = pointer && value ? PyTuple_Pack(2, pointer, value) : nullptr;
  Py_XDECREF(pointer);
  Py_XDECREF(value);
  return both;
}

PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t count) {
  long long n, width;
  if (count == 4 && THPVariable_Check(args[0]) && THPDtype_Check(args[1]) && number(args[2], &n) && number(args[3], &width)) {
    try {
      const at::Tensor& x = THPVariable_Unpack(args[0]);
      if (of_type(x, args[1]) && here(x) && x.dim() == 2 && x.size(0) >= n && x.size(1) >= width && x.stride(1) == 1)
        return pair(x.data_ptr(), x.stride(0));
    } catch (...) {
    }
  }
  Py_RETURN_NONE;
}

PyObject* states(PyObject*, PyObject* const* args, Py_ssize_t count) {
  long long want[3];
  if (count == 4 && THPVariable_Check(args[0]) && number(args[1], want) && number(args[2], want + 1) && number(args[3], want + 2)) {
    try {
      const at::Tensor& x = THPVariable_Unpack(args[0]);
      if (x.scalar_type() == at::kFloat && here(x) && x.dim() == 4 && x.size(1) == want[0] && x.size(2) == want[1] &&
          x.size(3) == want[2] && x.is_contiguous())
        return pair(x.data_ptr(), x.size(0));
    } catch (...) {
    }
  }
  Py_RETURN_NONE;
}

PyObject* otherwise(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(other, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"arg", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(arg)), METH_FASTCALL, nullptr},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rows)), METH_FASTCALL, nullptr},
    {"states", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(states)), METH_FASTCALL, nullptr},
    {"place", place, METH_O, nullptr},
    {"otherwise", otherwise, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host_args() { return PyModule_Create(&module); }
