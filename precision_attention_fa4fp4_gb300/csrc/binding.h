// binding.h -- what the native Python binding's calls share: argument parsing,
// checks of tensors, launches and errors.
#pragma once
#include <Python.h>
#include <structmember.h>

#include <ATen/ATen.h>
#include <ATen/Context.h>
#include <ATen/EmptyTensor.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fa4fp4.h"

namespace {

PyObject* g_error = nullptr;                 // Fa4Fp4Error(where, status)

// ---------------------------------------------------------------- arguments
struct Refused {};                           // a Python exception is set

[[noreturn]] void refuse(const char* format, ...) {
  va_list va;
  va_start(va, format);
  PyErr_FormatV(PyExc_ValueError, format, va);
  va_end(va);
  throw Refused();
}

// Up to 15 arguments by position or name; those not given are nullptr.
struct Signature {
  const char* where;
  int n, required;
  const char* names[15];
};

void parse(const Signature& s, PyObject* const* args, Py_ssize_t npos, PyObject* kw, PyObject** out) {
  for (int i = 0; i < s.n; ++i) out[i] = nullptr;
  if (npos > s.n) {
    PyErr_Format(PyExc_TypeError, "%s() takes %d arguments but %zd were given", s.where, s.n, npos);
    throw Refused();
  }
  for (Py_ssize_t i = 0; i < npos; ++i) out[i] = args[i];
  const Py_ssize_t nkw = kw ? PyTuple_GET_SIZE(kw) : 0;
  for (Py_ssize_t k = 0; k < nkw; ++k) {
    PyObject* name = PyTuple_GET_ITEM(kw, k);
    int i = 0;
    while (i < s.n && PyUnicode_CompareWithASCIIString(name, s.names[i]) != 0) ++i;
    if (i == s.n || out[i]) {
      PyErr_Format(PyExc_TypeError, "%s() got %s argument '%U'", s.where,
                   i == s.n ? "an unexpected keyword" : "multiple values for", name);
      throw Refused();
    }
    out[i] = args[npos + k];
  }
  for (int i = 0; i < s.required; ++i)
    if (!out[i]) {
      PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", s.where, s.names[i]);
      throw Refused();
    }
}

bool given(PyObject* x) { return x && x != Py_None; }

int as_int(PyObject* x, const char* name) {
  const long long v = PyLong_AsLongLong(x);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v < INT_MIN || v > INT_MAX) refuse("%s: out of range", name);
  return (int)v;
}

bool as_bool(PyObject* x, bool otherwise) {
  if (!x) return otherwise;
  const int v = PyObject_IsTrue(x);
  if (v < 0) throw Refused();
  return v != 0;
}

float as_float(PyObject* x) {
  if (!x) return 0.f;
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

const at::Tensor& as_tensor(PyObject* x, const char* name) {
  if (!THPVariable_Check(x)) refuse("%s: expected a tensor, got %s", name, Py_TYPE(x)->tp_name);
  return THPVariable_Unpack(x);
}

int64_t dim(const at::Tensor& t, const char* name, int dims, int i) {
  if (t.dim() != dims) refuse("%s: expected %d dimensions, got %d", name, dims, (int)t.dim());
  return t.size(i);
}

// A contiguous tensor of this shape and type on CUDA device `index`.
const at::Tensor& expect(PyObject* x, const char* name, int index, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor& t = as_tensor(x, name);
  if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) {
    std::string want = "[";
    for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
    refuse("%s: expected a contiguous %s tensor of shape %s] on cuda:%d", name, at::toString(type), want.c_str(), index);
  }
  return t;
}

int* ints(PyObject* x, const char* name, int index, at::IntArrayRef shape) {
  return given(x) ? static_cast<int*>(expect(x, name, index, at::kInt, shape).data_ptr()) : nullptr;
}

// Does anything look at the tensors that torch makes: a dispatch or function mode, a transform, or the filling of
// uninitialised memory?
bool watched() {
  const c10::DispatchKeySet keys = c10::impl::tls_local_dispatch_key_set().included_;
  const at::Context& torch = at::globalContext();
  return !(keys - c10::default_included_set).empty() ||
         (torch.deterministicAlgorithms() && torch.deterministicFillUninitializedMemory());
}

// A tensor of the caching allocator, made without the dispatcher where nothing there would see it: about 1 us
// instead of at::empty's 1.8, where a call makes up to five.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index, bool zero = false) {
  const at::TensorOptions how = at::TensorOptions().dtype(type).device(at::kCUDA, index);
  if (zero) return at::zeros(shape, how);
  if (watched()) return at::empty(shape, how);
  const int now = c10::cuda::current_device();
  if (now != index) c10::cuda::set_device((c10::DeviceIndex)index);
  struct Back {
    int now, index;
    ~Back() {
      if (now != index) c10::cuda::set_device((c10::DeviceIndex)now);
    }
  } back{now, index};
  return at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(),
                                   c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
}

// The caller's workspace, or a fresh one of `need` bytes (none for 0).
at::Tensor workspace(PyObject* x, int index, size_t need) {
  if (!given(x)) return need ? fresh({(int64_t)need}, at::kByte, index) : at::Tensor();
  const at::Tensor& t = as_tensor(x, "workspace");
  if (t.scalar_type() != at::kByte || !t.is_cuda() || t.get_device() != index || !t.is_contiguous())
    refuse("workspace: expected a contiguous uint8 tensor on the call's device");
  return t;
}

// ---------------------------------------------------------------- calls
// Runs `call(stream)` with device `index` current, without the interpreter lock.
template <class F>
void launch(const char* where, int index, F call) {
  const int now = c10::cuda::current_device();
  void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  if (now != index) c10::cuda::set_device((c10::DeviceIndex)index);
  fa4fp4_status status;
  Py_BEGIN_ALLOW_THREADS
  status = call(stream);
  Py_END_ALLOW_THREADS
  if (now != index) c10::cuda::set_device((c10::DeviceIndex)now);
  if (status != FA4FP4_OK) {
    PyObject* e = PyObject_CallFunction(g_error, "si", where, (int)status);
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    throw Refused();
  }
}

template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define FA4_METHOD(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS

}  // namespace
