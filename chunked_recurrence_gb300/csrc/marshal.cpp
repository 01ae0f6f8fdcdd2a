// marshal.cpp -- what the paged operators' Python binding does on every call, in C++: a key of its tensors'
// layouts (the checks of a layout run once, when its key is new) and its outputs.  A call's host time is a
// third less than with the same in Python, which the binding falls back to where this module is not built.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

namespace {

constexpr int kMost = 256, kDims = 8;  // tensors of a call (a fork's pools), dimensions of a tensor

// lays(*tensors) -> bytes: dtype, device, sizes and strides of each (None: absent)
PyObject *lays(PyObject *, PyObject *const *args, Py_ssize_t n) try {
  int64_t buf[kMost * (1 + 2 * kDims)];
  size_t k = 0;
  if (n > kMost) {
    PyErr_SetString(PyExc_ValueError, "too many tensors");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (args[i] == Py_None) {
      buf[k++] = -1;
      continue;
    }
    if (!THPVariable_Check(args[i])) {
      PyErr_SetString(PyExc_TypeError, "a tensor or None expected");
      return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    const int64_t d = t.dim();
    if (d > kDims) {
      PyErr_SetString(PyExc_ValueError, "too many dimensions");
      return nullptr;
    }
    buf[k++] = d | (int64_t)t.scalar_type() << 8 | (int64_t)t.device().type() << 16 | (int64_t)t.device().index() << 32;
    const auto size = t.sizes(), stride = t.strides();
    for (int64_t j = 0; j < d; ++j) buf[k++] = size[j], buf[k++] = stride[j];
  }
  return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(buf), k * sizeof(int64_t));
} catch (const std::exception &e) {  // a tensor without strides
  PyErr_SetString(PyExc_RuntimeError, e.what());
  return nullptr;
}

// like(tensor, dims, f32) -> a new contiguous tensor of the sizes of its first `dims` dimensions
PyObject *like(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 3 || !THPVariable_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "like(tensor, dims, f32)");
    return nullptr;
  }
  const at::Tensor &t = THPVariable_Unpack(args[0]);
  const long dims = PyLong_AsLong(args[1]);
  if (dims < 0 || dims > t.dim()) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "dims");
    return nullptr;
  }
  try {
    const auto options = args[2] == Py_True ? t.options().dtype(at::kFloat) : t.options();
    return THPVariable_Wrap(at::empty(t.sizes().slice(0, dims), options.requires_grad(false)));
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"lays", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(lays)), METH_FASTCALL, "key of layouts"},
    {"like", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(like)), METH_FASTCALL, "new tensor"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn_marshal", "paged operators' marshalling", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_gdn_marshal() {
  PyObject *m = PyModule_Create(&module);
  if (m) PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION);
  return m;
}
