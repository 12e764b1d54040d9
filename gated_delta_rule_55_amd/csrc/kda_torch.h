// kda_torch.h -- what the native modules on top of the library share: arguments read from
// Python objects, outputs, and the library's answers (see kda_torch.cpp for what they are
// for and what a function of theirs promises).
#pragma once

#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <utility>

#include "kda_norm.h"

namespace {

// Lets other Python threads run: around allocations and the library's calls,
// both of which may wait for the device.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  NoGil() = default;
  NoGil(const NoGil&) = delete;
  ~NoGil() { PyEval_RestoreThread(state); }
};

// A dense tensor argument of one device and type; `ok` turns false at the first
// argument that is none.
struct Args {
  bool ok = true;
  c10::DeviceIndex dev = -1;
  at::ScalarType dt = at::kFloat;

  const at::Tensor* tensor(PyObject* o) {
    if (!ok || !THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    // a plain tensor in memory: no lazy, functional or other wrapper
    ok = t.is_cuda() && t.layout() == at::kStrided && t.has_storage() && t.is_contiguous();
    return ok ? &t : nullptr;
  }
  // The same for a tensor whose rows or heads may lie apart.
  const at::Tensor* strided(PyObject* o) {
    if (!ok || !THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    ok = t.is_cuda() && t.layout() == at::kStrided && t.has_storage();
    return ok ? &t : nullptr;
  }
  // The tensor that sets device and type of the call.
  const at::Tensor* first(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    dev = t->device().index();
    dt = t->scalar_type();
    ok = (dt == at::kFloat || dt == at::kBFloat16) && dev == c10::hip::current_device();
    return ok ? t : nullptr;
  }
  void* ptr(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    ok = t->scalar_type() == type && t->device().index() == dev && t->sizes() == shape;
    return ok ? t->data_ptr() : nullptr;
  }
  void* maybe(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : ptr(o, type, shape);
  }
  float number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return (float)x;
  }
  // A scale: 0, the default's value, where there is none and for 0 alone.
  float scale(PyObject* o) {
    if (o == Py_None) return 0.f;
    const float x = number(o);
    if (x == 0.f && flag(o)) ok = false;
    return x;
  }
  bool flag(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) {
      PyErr_Clear();
      ok = false;
    }
    return x > 0;
  }
  int gate(PyObject* o) {
    if (o == Py_None) return KDA_NORM_GATE_LINEAR;
    if (PyUnicode_Check(o)) {
      if (PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0) return KDA_NORM_GATE_SIGMOID;
      if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return KDA_NORM_GATE_SILU;
      if (PyUnicode_CompareWithASCIIString(o, "none") == 0) return KDA_NORM_GATE_LINEAR;
    }
    ok = false;
    return 0;
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    const NoGil no_gil;
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, dev)));
  }
  // `o`'s tensor, or a new one where it is None; `made` then holds it.
  void* output(PyObject* o, at::ScalarType type, at::IntArrayRef shape, at::Tensor& made) {
    if (o != Py_None) return ptr(o, type, shape);
    if (!ok) return nullptr;
    made = empty(shape, type);
    return made.data_ptr();
  }
  void* stream() const { return c10::hip::getCurrentHIPStream(dev).stream(); }
};

inline int type_of(at::ScalarType t) { return t == at::kBFloat16 ? KDA_DTYPE_BF16 : KDA_DTYPE_F32; }

// An owned reference, or none.
struct Ref {
  PyObject* p = nullptr;
  Ref() = default;
  explicit Ref(PyObject* owned) : p(owned) {}
  Ref(Ref&& o) noexcept : p(o.release()) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* release() { return std::exchange(p, nullptr); }
};

inline Ref wrap(PyObject* given, at::Tensor& made) {
  if (made.defined()) return Ref(THPVariable_Wrap(std::move(made)));
  Py_INCREF(given);
  return Ref(given);
}

inline Ref pair(const Ref& a, const Ref& b) { return Ref(a.p && b.p ? PyTuple_Pack(2, a.p, b.p) : nullptr); }

// `result` when the library took the call, None when its checks refused it, and
// KdaError when a launch failed, after which part of the call may run.
inline PyObject* answer(int status, const char* what, Ref& result) {
  if (status == KDA_OK) return result.release();
  if (status != KDA_ERR_HIP) Py_RETURN_NONE;
  const Ref module(PyImport_ImportModule("gated_delta_rule_55_amd._abi"));
  const Ref type(module.p ? PyObject_GetAttrString(module.p, "KdaError") : nullptr);
  const Ref error(type.p ? PyObject_CallFunction(type.p, "is", status, what) : nullptr);
  if (error.p) PyErr_SetObject(type.p, error.p);
  return nullptr;
}

template <typename F>
int unlocked(F call) {
  const NoGil no_gil;
  return call();
}

// Runs f, with None for everything it throws, which is before its call of the
// library.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

}  // namespace
