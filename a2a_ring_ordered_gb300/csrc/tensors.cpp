// tensors.cpp -- addresses and sizes of a list of rank buffers, for ccl.py.
//
// A call names p tensors for each of its arguments.  Asking each of them for
// its dtype, device, size and address through Python takes half a microsecond
// a tensor, for eight ranks several times the launch itself; here it is a few
// loads.  ranks() and shaped() return None for anything that is not as the
// caller wants it, and the caller then finds out what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <cstring>
#include <exception>
#include <vector>

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

// on_device(device, lists) -> whether the first tensor of every list in a tuple
// of lists (None: no list) is on that GPU; None where one is no such list.
PyObject* on_device(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2 || !PyTuple_CheckExact(args[1])) return PyErr_Format(PyExc_TypeError, "on_device() takes a number and a tuple of lists");
  const Py_ssize_t device = PyLong_AsSsize_t(args[0]);
  if (PyErr_Occurred() != nullptr) return nullptr;
  try {
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(args[1]); ++i) {
      PyObject* ts = PyTuple_GET_ITEM(args[1], i);
      if (ts == Py_None) continue;
      if (length(ts) < 0 || !THPVariable_Check(PySequence_Fast_GET_ITEM(ts, 0))) Py_RETURN_NONE;
      const at::Tensor& t = THPVariable_Unpack(PySequence_Fast_GET_ITEM(ts, 0));
      if (!t.defined() || !t.is_cuda() || t.get_device() != device) Py_RETURN_FALSE;
    }
  } catch (...) {
    Py_RETURN_NONE;
  }
  Py_RETURN_TRUE;
}

// Where a tensor's elements are, and which.
struct Place {
  const void* data;  // of its storage
  int64_t offset, numel;
  uint64_t kind;
};
inline Place place_of(const c10::TensorImpl* t) {
  return {t->unsafe_storage().unsafeGetStorageImpl()->data(), t->storage_offset(), t->numel(),
          static_cast<uint64_t>(c10::typeMetaToScalarType(t->dtype())) << 1 | static_cast<uint64_t>(t->is_contiguous())};
}

// Calls f(tensor, its number) for the items of a tuple of tuples.
template <typename F>
void each_item(PyObject* tuples, F f) {
  Py_ssize_t k = 0;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tuples); ++i) {
    PyObject* ts = PyTuple_GET_ITEM(tuples, i);
    for (Py_ssize_t j = 0; j < PyTuple_GET_SIZE(ts); ++j) f(PyTuple_GET_ITEM(ts, j), k++);
  }
}

// places(tuples) -> the places of the tensors in a tuple of tuples, as bytes.
PyObject* places(PyObject*, PyObject* tuples) {
  bool ok = PyTuple_CheckExact(tuples);
  for (Py_ssize_t i = 0; ok && i < PyTuple_GET_SIZE(tuples); ++i) ok = PyTuple_CheckExact(PyTuple_GET_ITEM(tuples, i));
  Py_ssize_t count = 0;
  if (ok)
    each_item(tuples, [&](PyObject* o, Py_ssize_t) {
      ok = ok && THPVariable_Check(o) && THPVariable_Unpack(o).defined() && THPVariable_Unpack(o).has_storage();
      ++count;
    });
  if (!ok) return PyErr_Format(PyExc_TypeError, "places() takes a tuple of tuples of tensors");
  std::vector<Place> out(static_cast<size_t>(count));
  try {
    each_item(tuples, [&](PyObject* o, Py_ssize_t k) { out[static_cast<size_t>(k)] = place_of(THPVariable_Unpack(o).unsafeGetTensorImpl()); });
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_ValueError, "%s", e.what());
  }
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(out.data()), count * static_cast<Py_ssize_t>(sizeof(Place)));
}

// in_place(tuples, places) -> whether the tensors of places(tuples), the same
// tuples as then, are where they were: 5 to 7 ns a tensor.
PyObject* in_place(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2 || !PyTuple_CheckExact(args[0]) || !PyBytes_CheckExact(args[1])) return PyErr_Format(PyExc_TypeError, "in_place() takes a tuple and bytes");
  const char* was = PyBytes_AS_STRING(args[1]);
  const Py_ssize_t held = PyBytes_GET_SIZE(args[1]) / static_cast<Py_ssize_t>(sizeof(Place));
  bool same = true;
  try {
    each_item(args[0], [&](PyObject* o, Py_ssize_t k) {
      if (k >= held) {
        same = false;
        return;
      }
      Place old;
      memcpy(&old, was + k * static_cast<Py_ssize_t>(sizeof(Place)), sizeof(old));
      const Place now = place_of(THPVariable_Unpack(o).unsafeGetTensorImpl());
      same &= now.data == old.data && now.offset == old.offset && now.numel == old.numel && now.kind == old.kind;
    });
  } catch (...) {  // a storage that has no data to point at
    same = false;
  }
  return PyBool_FromLong(same);
}

PyMethodDef methods[] = {
    {"places", places, METH_O, nullptr},
    {"in_place", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(in_place)), METH_FASTCALL, nullptr},
    {"on_device", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(on_device)), METH_FASTCALL, nullptr},
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
