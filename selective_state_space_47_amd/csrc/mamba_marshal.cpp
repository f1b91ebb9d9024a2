// mamba_marshal.cpp -- the per-call part of the Python binding: what a call's tensors look like, as one
// bytes object, and their addresses handed to the C entry point.  Checks, allocation and errors stay in
// binding.py; it looks a call's key up in a cache of keys that have passed the checks.  A launch of a few
// microseconds (one token, one row) would otherwise be dominated by reading tensors' metadata from Python:
// 9 to 10 us a call against 5.
#include <Python.h>
#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "mamba_scan.h"

namespace {

template <typename T>
void put(std::string& s, T v) {
  s.append(reinterpret_cast<const char*>(&v), sizeof(v));
}

// key(*args) -> bytes.  Two argument lists with the same key have the same types, shapes, strides, devices
// and small values; only addresses and contents differ.  A tensor without sizes or strides (a nested one)
// raises, and so does one whose values are not those in its memory.
PyObject* key(PyObject*, PyObject* const* args, Py_ssize_t n) try {
  std::string s;
  s.reserve(64 * n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = args[i];
    if (o == Py_None) {
      s += 'N';
    } else if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.layout() != at::kStrided) {
        s += 'L';  // (the checks refuse it: it has no strides)
        continue;
      }
      if (t.is_neg()) {
        PyErr_SetString(PyExc_ValueError, "a tensor of the call is a lazily negated view: pass its resolve_neg()");
        return nullptr;
      }
      s += 'T';
      put(s, (int8_t)t.scalar_type());
      put(s, (int8_t)t.device().type());
      put(s, (int8_t)t.device().index());
      put(s, (int8_t)t.dim());
      for (int64_t v : t.sizes()) put(s, v);
      for (int64_t v : t.strides()) put(s, v);
    } else if (PyBool_Check(o)) {
      s += o == Py_True ? '1' : '0';
    } else if (PyLong_Check(o)) {
      int over = 0;
      s += 'I';
      put(s, (int64_t)PyLong_AsLongLongAndOverflow(o, &over));
      put(s, (int8_t)over);
    } else {
      s += 'O';  // of a type that the checks refuse
      put(s, Py_TYPE(o));
    }
  }
  return PyBytes_FromStringAndSize(s.data(), (Py_ssize_t)s.size());
} catch (const c10::Error& e) {  // (not torch's macro around it: that has a cost where nothing is thrown)
  PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  return nullptr;
} catch (const std::exception& e) {
  PyErr_SetString(PyExc_RuntimeError, e.what());
  return nullptr;
}

void* address(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw std::invalid_argument("a tensor or None");
  return THPVariable_Unpack(o).data_ptr();
}

// empty(like) -> a new contiguous tensor of like's shape, type and device
// empty(like, type, *sizes) -> of these sizes on like's device, type 'f' (float32) or 'b' (bytes)
// 0.9 us; like.new_empty(like.shape) from Python takes 1.8.
PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 1 || n > 6 || !THPVariable_Check(args[0]) || (n > 1 && !PyUnicode_Check(args[1]))) {
    PyErr_SetString(PyExc_TypeError, "empty(like) or empty(like, type, up to four sizes)");
    return nullptr;
  }
  HANDLE_TH_ERRORS  // (out of memory is torch's own error)
  const at::Tensor& like = THPVariable_Unpack(args[0]);
  int64_t dims[4];
  at::IntArrayRef sizes = like.sizes();
  at::ScalarType type = like.scalar_type();
  if (n > 1) {
    for (Py_ssize_t i = 2; i < n; ++i) dims[i - 2] = PyLong_AsLongLong(args[i]);
    if (PyErr_Occurred()) return nullptr;
    sizes = at::IntArrayRef(dims, n - 2);
    type = PyUnicode_ReadChar(args[1], 0) == 'f' ? at::kFloat : at::kByte;
  }
  return THPVariable_Wrap(at::empty(sizes, like.options().dtype(type)));
  END_HANDLE_TH_ERRORS
}

enum Entry { kDeltaFwd, kDeltaUpdate, kDeltaBwd, kGatedFwd, kGatedBwd, kAddFwd, kAddBwd };

// call(entry, dims address, stream, factor, workspace bytes, *tensors) -> status.  The tensors stand in the
// order of the entry point's pointers, `factor` is its scale or eps.
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 5 || n > 25) {
    PyErr_SetString(PyExc_TypeError, "call(entry, dims, stream, factor, workspace bytes, *tensors)");
    return nullptr;
  }
  const long entry = PyLong_AsLong(args[0]);
  void* d = PyLong_AsVoidPtr(args[1]);
  void* stream = PyLong_AsVoidPtr(args[2]);
  const float f = (float)PyFloat_AsDouble(args[3]);
  const size_t ws = PyLong_AsSize_t(args[4]);
  if (PyErr_Occurred()) return nullptr;
  void* p[20] = {};
  try {
    for (Py_ssize_t i = 5; i < n; ++i) p[i - 5] = address(args[i]);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
    return nullptr;
  }
  auto fp = [&](int i) { return static_cast<float*>(p[i]); };
  static const int kTensors[] = {10, 7, 16, 4, 8, 7, 13};
  if (entry < kDeltaFwd || entry > kAddBwd || n - 5 != kTensors[entry]) {
    PyErr_SetString(PyExc_TypeError, "wrong number of tensors for the entry point");
    return nullptr;
  }
  int st = 0;
  // (a launch waits where the queue is full: other Python threads go on meanwhile)
  Py_BEGIN_ALLOW_THREADS
  switch (entry) {
    case kDeltaFwd:
      st = mamba_delta_fwd(p[0], p[1], p[2], p[3], p[4], fp(5), static_cast<int64_t*>(p[6]), f, p[7], fp(8),
                           static_cast<mamba_delta_dims*>(d), p[9], ws, stream);
      break;
    case kDeltaUpdate:
      st = mamba_delta_update(fp(0), p[1], p[2], p[3], p[4], p[5], f, p[6],
                              static_cast<mamba_delta_dims*>(d), stream);
      break;
    case kDeltaBwd:
      st = mamba_delta_bwd(p[0], p[1], p[2], p[3], p[4], fp(5), static_cast<int64_t*>(p[6]), f, p[7], fp(8),
                           p[9], p[10], p[11], p[12], p[13], fp(14), static_cast<mamba_delta_dims*>(d), p[15],
                           ws, stream);
      break;
    case kGatedFwd:
      st = mamba_gated_norm_fwd(p[0], p[1], fp(2), f, p[3], static_cast<mamba_gated_norm_dims*>(d), stream);
      break;
    case kGatedBwd:
      st = mamba_gated_norm_bwd(p[0], p[1], fp(2), f, p[3], p[4], p[5], fp(6),
                                static_cast<mamba_gated_norm_dims*>(d), p[7], ws, stream);
      break;
    case kAddFwd:
      st = mamba_add_norm_fwd(p[0], p[1], fp(2), fp(3), fp(4), f, p[5], p[6],
                              static_cast<mamba_add_norm_dims*>(d), stream);
      break;
    case kAddBwd:
      st = mamba_add_norm_bwd(p[0], p[1], fp(2), fp(3), fp(4), f, p[5], p[6], p[7], p[8], fp(9), fp(10), fp(11),
                              static_cast<mamba_add_norm_dims*>(d), p[12], ws, stream);
      break;
  }
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

PyMethodDef kMethods[] = {
    {"key", (PyCFunction)(void (*)())key, METH_FASTCALL, "key(*args) -> bytes: types, shapes, strides, devices"},
    {"call", (PyCFunction)(void (*)())call, METH_FASTCALL,
     "call(entry, dims address, stream, factor, workspace bytes, *tensors) -> status"},
    {"empty", (PyCFunction)(void (*)())empty, METH_FASTCALL, "empty(like[, type, *sizes]) -> a new contiguous tensor"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "mamba_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the headers that this was compiled against, which the binding compares with the torch it has
PyMODINIT_FUNC PyInit_mamba_marshal(void) {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "torch_version", MAMBA_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
