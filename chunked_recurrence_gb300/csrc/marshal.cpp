// marshal.cpp -- what the paged operators' Python binding does on every call, in C++: a key of its tensors'
// layouts (the checks of a layout run once, when its key is new), its outputs, and the library call itself.
// The binding does the same in Python where this module is not built, at twice the host time a call.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/Allocator.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <algorithm>
#include <cstring>
#include <tuple>
#include <type_traits>

#include "gdn.h"

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

struct PyRaised {};  // a Python error has been set

// The exception being handled as Python's; nullptr.
PyObject *raised() {
  try {
    throw;
  } catch (const PyRaised &) {
  } catch (const c10::OutOfMemoryError &e) {  // what torch's own allocations raise
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// One argument of a library call: a pointer is a tensor's data, a bytes object's, an address or None.
template <typename P>
P argument(PyObject *o) {
  if constexpr (std::is_pointer_v<P>) {
    if (o == Py_None) return nullptr;
    if (THPVariable_Check(o)) return (P)THPVariable_Unpack(o).data_ptr();
    if (PyBytes_Check(o)) return (P)PyBytes_AS_STRING(o);
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PyRaised{};
    return (P)p;
  } else if constexpr (std::is_floating_point_v<P>) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw PyRaised{};
    return (P)x;
  } else {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw PyRaised{};
    if ((P)x != x) {
      PyErr_SetString(PyExc_OverflowError, "an argument does not fit its type");
      throw PyRaised{};
    }
    return (P)x;
  }
}

// pack(tail, *pointers) -> bytes: the pointers (as in a call), then the bytes of tail: a struct of the library
PyObject *pack(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n < 1 || n > kMost + 1 || !PyBytes_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "pack(tail, *pointers)");
    return nullptr;
  }
  const Py_ssize_t heads = (n - 1) * sizeof(void *), tail = PyBytes_GET_SIZE(args[0]);
  PyObject *out = PyBytes_FromStringAndSize(nullptr, heads + tail);
  if (!out) return nullptr;
  char *p = PyBytes_AS_STRING(out);
  memcpy(p + heads, PyBytes_AS_STRING(args[0]), tail);
  try {
    for (Py_ssize_t i = 1; i < n; ++i, p += sizeof(void *)) {
      const void *x = argument<void *>(args[i]);
      memcpy(p, &x, sizeof x);
    }
    return out;
  } catch (...) {
    Py_DECREF(out);
    return raised();
  }
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
  } catch (...) {
    return raised();
  }
}

// Calls f.  SCRATCH: its workspace (the third last argument, its size the second last), where it is None, is memory of
// the current stream for this call: given back as the call returns, for what the stream does next.
template <bool SCRATCH, typename... P, size_t... I>
gdn_status invoke(gdn_status (*f)(P...), PyObject *const *args, std::index_sequence<I...>) {
  std::tuple<P...> a{argument<P>(args[I])...};
  at::DataPtr scratch;
  if constexpr (SCRATCH) {
    constexpr size_t kAt = sizeof...(P) - 3;
    if (!std::get<kAt>(a)) {
      size_t &bytes = std::get<kAt + 1>(a);
      bytes = std::max<size_t>(bytes, 256);
      scratch = c10::GetAllocator(c10::DeviceType::CUDA)->allocate(bytes);
      std::get<kAt>(a) = scratch.get();
    }
  }
  PyThreadState *state = PyEval_SaveThread();
  const gdn_status st = f(std::get<I>(a)...);
  PyEval_RestoreThread(state);
  return st;
}

template <typename F, bool SCRATCH>
struct Entry;
// call(address of the library's function, its arguments) -> status
template <typename... P, bool SCRATCH>
struct Entry<gdn_status(P...), SCRATCH> {
  static PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 1 + (Py_ssize_t)sizeof...(P)) {
      PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
      return nullptr;
    }
    try {
      auto *f = (gdn_status(*)(P...))argument<void *>(args[0]);
      return PyLong_FromLong(invoke<SCRATCH>(f, args + 1, std::index_sequence_for<P...>{}));
    } catch (...) {
      return raised();
    }
  }
};

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

#define GDN_ENTRY(name) {#name, fast(Entry<decltype(name), false>::call), METH_FASTCALL, "library call"}
#define GDN_ENTRY_SCRATCH(name) {#name, fast(Entry<decltype(name), true>::call), METH_FASTCALL, "library call"}
PyMethodDef methods[] = {
    {"lays", fast(lays), METH_FASTCALL, "key of layouts"},
    {"like", fast(like), METH_FASTCALL, "new tensor"},
    {"pack", fast(pack), METH_FASTCALL, "struct of pointers and a tail"},
    GDN_ENTRY(gdn_rope),
    GDN_ENTRY(gdn_kv_append),
    GDN_ENTRY_SCRATCH(gdn_paged_attn),
    GDN_ENTRY_SCRATCH(gdn_paged_attn_shared),
    GDN_ENTRY_SCRATCH(gdn_paged_mass),
    GDN_ENTRY_SCRATCH(gdn_pages_grow),
    GDN_ENTRY(gdn_pages_free),
    GDN_ENTRY_SCRATCH(gdn_pages_fork),
    GDN_ENTRY_SCRATCH(gdn_pages_compact),
    GDN_ENTRY(gdn_pages_copy),
    GDN_ENTRY_SCRATCH(gdn_pages_evict),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn_marshal", "paged operators' marshalling", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_gdn_marshal() {
  PyObject *m = PyModule_Create(&module);
  if (m) PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION);
  return m;
}
