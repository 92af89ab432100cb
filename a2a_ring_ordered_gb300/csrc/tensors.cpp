// tensors.cpp -- addresses and sizes of a list of rank buffers, for ccl.py.
//
// A call names p tensors for each of its arguments.  Asking each of them for
// its dtype, device, size and address through Python takes half a microsecond
// a tensor, for eight ranks several times the launch itself; here it is a few
// loads.  Both functions return None for anything that is not as the caller
// wants it, and the caller then finds out what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>

namespace {

constexpr Py_ssize_t kMaxRanks = 128;  // CCL_MAX_RANKS

// The items of a list or tuple of 1 to kMaxRanks, or -1.
Py_ssize_t length(PyObject* ts) {
  if (!PyList_CheckExact(ts) && !PyTuple_CheckExact(ts)) return -1;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(ts);
  return n >= 1 && n <= kMaxRanks ? n : -1;
}

// The tensor at place i where it is a contiguous CUDA tensor, else null.
const at::Tensor* buffer_at(PyObject* ts, Py_ssize_t i) {
  PyObject* o = PySequence_Fast_GET_ITEM(ts, i);
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.defined() && t.is_cuda() && t.layout() == at::kStrided && t.is_contiguous() ? &t : nullptr;
}

// ranks(ts, p, dtype, rows, width) -> the addresses of p buffers of dtype on
// one device as bytes, buffer r of rows[r] * width elements.
PyObject* ranks(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) return PyErr_Format(PyExc_TypeError, "ranks() takes 5 arguments");
  const Py_ssize_t p = length(args[0]);
  if (p < 0 || !THPDtype_Check(args[2]) || !PyList_CheckExact(args[3]) || PyList_GET_SIZE(args[3]) != p) Py_RETURN_NONE;
  const Py_ssize_t want = PyLong_AsSsize_t(args[1]), width = PyLong_AsSsize_t(args[4]);
  if (PyErr_Occurred() != nullptr) return nullptr;
  if (want != p) Py_RETURN_NONE;
  const at::ScalarType type = reinterpret_cast<THPDtype*>(args[2])->scalar_type;
  uint64_t out[kMaxRanks];
  try {
    const at::Tensor* first = nullptr;
    for (Py_ssize_t r = 0; r < p; ++r) {
      const at::Tensor* t = buffer_at(args[0], r);
      if (first == nullptr) first = t;
      const Py_ssize_t rows = PyLong_AsSsize_t(PyList_GET_ITEM(args[3], r));
      if (rows == -1 && PyErr_Occurred() != nullptr) return nullptr;
      if (t == nullptr || t->scalar_type() != type || t->get_device() != first->get_device() || t->numel() != rows * width) Py_RETURN_NONE;
      out[r] = reinterpret_cast<uintptr_t>(t->data_ptr());
    }
  } catch (...) {  // a tensor without storage
    Py_RETURN_NONE;
  }
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(out), p * 8);
}

// shaped(ts, dims, p or None, dtype or None) -> (addresses, [first dimension of
// each], the other dimensions) of buffers of `dims` dimensions on one device,
// alike but for the first dimension.
PyObject* shaped(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4) return PyErr_Format(PyExc_TypeError, "shaped() takes 4 arguments");
  const Py_ssize_t p = length(args[0]), dims = PyLong_AsSsize_t(args[1]), want = args[2] == Py_None ? p : PyLong_AsSsize_t(args[2]);
  if (PyErr_Occurred() != nullptr) return nullptr;
  if (p < 0 || want != p || dims < 1 || (args[3] != Py_None && !THPDtype_Check(args[3]))) Py_RETURN_NONE;
  uint64_t out[kMaxRanks];
  int64_t sizes[kMaxRanks];
  const at::Tensor* first = nullptr;
  try {
    for (Py_ssize_t r = 0; r < p; ++r) {
      const at::Tensor* t = buffer_at(args[0], r);
      if (t == nullptr || t->dim() != dims) Py_RETURN_NONE;
      if (first == nullptr) {
        first = t;
        if (args[3] != Py_None && t->scalar_type() != reinterpret_cast<THPDtype*>(args[3])->scalar_type) Py_RETURN_NONE;
      }
      if (t->scalar_type() != first->scalar_type() || t->get_device() != first->get_device() ||
          t->sizes().slice(1) != first->sizes().slice(1))
        Py_RETURN_NONE;
      sizes[r] = t->size(0);
      out[r] = reinterpret_cast<uintptr_t>(t->data_ptr());
    }
  } catch (...) {
    Py_RETURN_NONE;
  }
  PyObject* list = PyList_New(p);
  PyObject* rest = PyTuple_New(dims - 1);
  PyObject* bytes = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(out), p * 8);
  PyObject* all = nullptr;
  bool ok = list != nullptr && rest != nullptr && bytes != nullptr;
  for (Py_ssize_t r = 0; ok && r < p; ++r) {
    PyObject* v = PyLong_FromLongLong(sizes[r]);
    ok = v != nullptr;
    if (ok) PyList_SET_ITEM(list, r, v);
  }
  for (Py_ssize_t d = 1; ok && d < dims; ++d) {
    PyObject* v = PyLong_FromLongLong(first->size(d));
    ok = v != nullptr;
    if (ok) PyTuple_SET_ITEM(rest, d - 1, v);
  }
  if (ok) all = PyTuple_Pack(3, bytes, list, rest);
  Py_XDECREF(list);
  Py_XDECREF(rest);
  Py_XDECREF(bytes);
  return all;
}

PyMethodDef methods[] = {
    {"ranks", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ranks)), METH_FASTCALL, nullptr},
    {"shaped", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(shaped)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__tensors() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "TORCH_VERSION", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
