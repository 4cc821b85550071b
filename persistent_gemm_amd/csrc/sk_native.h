// What the native binding's calls share: arguments, outputs, streams and errors.
#pragma once

#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/DeviceGuardImplInterface.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../include/sk_gemm.h"

namespace sk_native {

using at::Tensor;

// An argument: a tensor, None, or neither.
struct Arg {
  const Tensor* t = nullptr;
  bool bad = false;
  explicit Arg(PyObject* o) {
    if (THPVariable_Check(o)) t = &THPVariable_Unpack(o);
    else bad = o != Py_None;
  }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
};

inline bool is(const Tensor& t, c10::Device dev, at::ScalarType type, at::IntArrayRef shape) {
  return t.layout() == at::kStrided && t.device() == dev && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous();
}
// NULL, or as described.
inline bool none_or(const Arg& a, c10::Device dev, at::ScalarType type, at::IntArrayRef shape) {
  return !a.bad && (!a.t || is(*a.t, dev, type, shape));
}

// An output, from the allocator that torch's own tensors of the device come from (the first one says which).  at::empty
// finds it through two dispatches: 0.75 us a tensor against 0.32.  The allocator serves the current device, which
// stream_of() has made sure of.
inline Tensor make(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  static c10::Allocator* allocator = nullptr;
  if (allocator) return at::detail::empty_generic(shape, allocator, c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
  const Tensor t = at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  allocator = t.storage().allocator();
  return t;
}

// The stream to use: the caller's handle, or torch's current one of the device (by the function bind() was given).
// False where the handle is none, or the device not the current one, which the library launches on.
extern PyObject* current_stream;
inline bool stream_of(PyObject* o, c10::Device dev, void** s) {
  if (c10::impl::getDeviceGuardImpl(dev.type())->getDevice() != dev) return false;
  if (o == Py_None) {
    PyObject* index = PyLong_FromLong(dev.index());
    PyObject* handle = index ? PyObject_CallFunctionObjArgs(current_stream, index, nullptr) : nullptr;
    *s = handle ? PyLong_AsVoidPtr(handle) : nullptr;
    Py_XDECREF(index);
    Py_XDECREF(handle);
  } else {
    *s = PyLong_AsVoidPtr(o);
  }
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

inline PyObject* put(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
inline PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  if (r)
    for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, put(t));
  return r;
}
inline PyObject* refuse() { Py_RETURN_NONE; }

// Whatever torch throws (out of memory, say) leaves as a Python error.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// The interpreter lock given up for a call that uses the library's scratch: it may wait for another thread's call on the
// stream, or for the stream itself when the scratch has to grow.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void*)F, METH_FASTCALL, nullptr};
}

// The calls of a layer of experts (sk_native_experts.cpp), up to a method without a name.
extern PyMethodDef experts_methods[];

}  // namespace sk_native
