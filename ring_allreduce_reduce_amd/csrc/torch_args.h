// What the functions of the torch binding share: arguments' checks, output
// tensors and refusals.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "ringar.h"

namespace ringar_torch {

struct Refusal {
  int code;
  std::string what;
};

[[noreturn]] inline void bad(const std::string& why) { throw Refusal{RINGAR_ERR_INVALID_ARGUMENT, why}; }

// A tensor argument, or null for None.
inline const at::Tensor* tensor(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad(std::string(what) + " must be a tensor");
  const at::Tensor* t = &THPVariable_Unpack(o);
  if (t->is_neg()) bad(std::string(what) + " is a negated view (call resolve_neg() first)");
  return t;
}

inline const at::Tensor& needed(PyObject* o, const char* what) {
  const at::Tensor* t = tensor(o, what);
  if (!t) bad(std::string(what) + " is needed");
  return *t;
}

inline int code_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return RINGAR_FLOAT16;
    case at::kBFloat16: return RINGAR_BFLOAT16;
    case at::kFloat: return RINGAR_FLOAT32;
    default: return -1;
  }
}

// The operand that the others go by: its type, its GPU, which becomes the
// current one for the call, and that GPU's current stream.
struct Call {
  const at::Tensor& of;
  at::ScalarType type;
  int code;
  c10::OptionalDeviceGuard guard;

  explicit Call(const at::Tensor& t, const char* what) : of(t), type(t.scalar_type()), code(code_of(type)) {
    if (!t.is_cuda()) bad(std::string(what) + " must be a CUDA tensor");
    if (code < 0) bad(std::string("unsupported dtype ") + at::toString(type) + ": float16, bfloat16 or float32");
    if (t.get_device() != c10::hip::current_device()) guard.reset_device(t.device());
  }
  ringar_stream_t stream() const { return (ringar_stream_t)c10::hip::getCurrentHIPStream(of.get_device()).stream(); }
  at::Tensor make(at::IntArrayRef sizes) const { return at::empty(sizes, of.options()); }
  at::Tensor make(at::IntArrayRef sizes, at::ScalarType t) const { return at::empty(sizes, of.options().dtype(t)); }
};

// Rows of a tensor whose last dimension is contiguous.
struct Rows {
  int64_t rows = 0, cols = 0, ld = 0;
  void* p = nullptr;

  Rows() = default;
  Rows(const at::Tensor& t, const char* what, const Call& call) {
    if (t.scalar_type() != call.type || !t.is_cuda() || t.get_device() != call.of.get_device())
      bad(std::string(what) + " must have the dtype and device of the other operands");
    const auto size = t.sizes(), stride = t.strides();
    const int64_t n = (int64_t)size.size();
    if (n == 0) bad(std::string(what) + " needs at least one dimension");
    p = t.data_ptr();
    cols = size[n - 1];
    if (cols > 1 && stride[n - 1] != 1) bad(std::string(what) + ": the last dimension must be contiguous");
    rows = 1;
    bool found = false;
    for (int64_t i = n - 2; i >= 0; i--) {
      if (size[i] == 0) {
        rows = 0;
        ld = cols;
        return;
      }
    }
    for (int64_t i = n - 2; i >= 0; i--) {
      if (size[i] == 1) continue;
      if (!found) {
        ld = stride[i];
        found = true;
      } else if (stride[i] != rows * ld) {
        bad(std::string(what) + ": the rows must lie at one stride (make the tensor contiguous first)");
      }
      rows *= size[i];
    }
    if (!found) ld = cols;
  }
};

inline void* vec(const at::Tensor* t, int64_t n, const char* what, at::ScalarType type, const Call& call) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || !t->is_cuda() || t->get_device() != call.of.get_device() || t->dim() != 1 || t->size(0) != n ||
      !t->is_contiguous())
    bad(std::string(what) + " must be a contiguous vector of " + std::to_string(n) + " values of " + at::toString(type) +
        " on the operands' GPU");
  return t->data_ptr();
}

inline c10::SmallVector<int64_t, 6> shape_of(const at::Tensor& like, int64_t last) {
  c10::SmallVector<int64_t, 6> s(like.sizes().begin(), like.sizes().end());
  s.back() = last;
  return s;
}

inline void done(int code, const char* name) {
  if (code != RINGAR_SUCCESS) throw Refusal{code, std::string(name) + " (" + ringar_last_error() + ")"};
}

inline PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

inline PyObject* wrap_or_none(at::Tensor t) {
  if (t.defined()) return wrap(std::move(t));
  Py_RETURN_NONE;
}

inline PyObject* tuple(std::initializer_list<PyObject*> v) {
  PyObject* r = PyTuple_New((Py_ssize_t)v.size());
  Py_ssize_t i = 0;
  for (PyObject* o : v) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

// A caller's tensor that the call has written: autograd must not take a value
// that it has kept of it for unchanged.  (Inference tensors are not counted.)
inline void written(const at::Tensor* t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

inline bool truth(PyObject* o, const char* what) {
  if (o != Py_True && o != Py_False) bad(std::string(what) + " must be True or False");
  return o == Py_True;
}
inline void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// torch_layer.cpp
PyObject* rms_norm(PyObject* const* v);
PyObject* rms_norm_backward(PyObject* const* v);
PyObject* dropout(PyObject* const* v);
PyObject* cross_attention(PyObject* const* v);
PyObject* cross_attention_backward(PyObject* const* v);

}  // namespace ringar_torch
