// The block operators on torch tensors: argument checks, output tensors and
// the C call, in one extension function each (a call of a few microseconds
// spends most of them here; the same checks in Python took 4 us more).
// Signatures, defaults and streams are block.py's.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "ringar.h"

namespace {

struct Refusal {
  int code;
  std::string what;
};

[[noreturn]] void bad(const std::string& why) { throw Refusal{RINGAR_ERR_INVALID_ARGUMENT, why}; }

// A tensor argument, or null for None.
const at::Tensor* tensor(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad(std::string(what) + " must be a tensor");
  const at::Tensor* t = &THPVariable_Unpack(o);
  if (t->is_neg()) bad(std::string(what) + " is a negated view (call resolve_neg() first)");
  return t;
}

const at::Tensor& needed(PyObject* o, const char* what) {
  const at::Tensor* t = tensor(o, what);
  if (!t) bad(std::string(what) + " is needed");
  return *t;
}

int code_of(at::ScalarType t) {
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

void* vec(const at::Tensor* t, int64_t n, const char* what, at::ScalarType type, const Call& call) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || !t->is_cuda() || t->get_device() != call.of.get_device() || t->dim() != 1 || t->size(0) != n ||
      !t->is_contiguous())
    bad(std::string(what) + " must be a contiguous vector of " + std::to_string(n) + " values of " + at::toString(type) +
        " on the operands' GPU");
  return t->data_ptr();
}

c10::SmallVector<int64_t, 6> shape_of(const at::Tensor& like, int64_t last) {
  c10::SmallVector<int64_t, 6> s(like.sizes().begin(), like.sizes().end());
  s.back() = last;
  return s;
}

void done(int code, const char* name) {
  if (code != RINGAR_SUCCESS) throw Refusal{code, std::string(name) + " (" + ringar_last_error() + ")"};
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

PyObject* wrap_or_none(at::Tensor t) {
  if (t.defined()) return wrap(std::move(t));
  Py_RETURN_NONE;
}

PyObject* tuple(std::initializer_list<PyObject*> v) {
  PyObject* r = PyTuple_New((Py_ssize_t)v.size());
  Py_ssize_t i = 0;
  for (PyObject* o : v) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

// A caller's tensor that the call has written: autograd must not take a value
// that it has kept of it for unchanged.  (Inference tensors are not counted.)
void written(const at::Tensor* t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

bool truth(PyObject* o, const char* what) {
  if (o != Py_True && o != Py_False) bad(std::string(what) + " must be True or False");
  return o == Py_True;
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject* layer_norm(PyObject* const* v) {
  const at::Tensor& x = needed(v[0], "x");
  const at::Tensor *weight = tensor(v[1], "weight"), *bias = tensor(v[2], "bias"), *out = tensor(v[5], "out");
  const double eps = PyFloat_AsDouble(v[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const bool stats = truth(v[4], "stats");
  Call call(x, "x");
  const Rows rx(x, "x", call);
  const at::ScalarType ptype = weight ? weight->scalar_type() : bias ? bias->scalar_type() : call.type;
  ringar_layer_norm_t a = {};
  a.dtype = (ringar_dtype_t)call.code;
  a.param_dtype = (ringar_dtype_t)code_of(ptype);
  a.rows = rx.rows;
  a.cols = rx.cols;
  a.x = rx.p;
  a.ldx = rx.ld;
  a.weight = vec(weight, rx.cols, "weight", ptype, call);
  a.bias = vec(bias, rx.cols, "bias", ptype, call);
  a.eps = (float)eps;
  at::Tensor y, mean, rstd;
  if (out) {
    if (out->sizes() != x.sizes()) bad("out must have x's shape");
    const Rows ry(*out, "out", call);
    y = *out;
    a.ldy = ry.ld;
  } else {
    y = call.make(x.sizes());
    a.ldy = rx.cols;
  }
  a.y = y.data_ptr();
  if (stats) {
    mean = call.make(x.sizes().slice(0, x.dim() - 1), at::kFloat);
    rstd = call.make(x.sizes().slice(0, x.dim() - 1), at::kFloat);
    a.mean = (float*)mean.data_ptr();
    a.rstd = (float*)rstd.data_ptr();
  }
  done(ringar_layer_norm(&a, call.stream()), "ringar_layer_norm");
  written(out);
  if (!stats) return wrap(y);
  return tuple({wrap(y), wrap(mean), wrap(rstd)});
}

PyObject* layer_norm_backward(PyObject* const* v) {
  const at::Tensor &dy = needed(v[0], "dy"), &x = needed(v[1], "x"), &mean = needed(v[2], "mean"), &rstd = needed(v[3], "rstd");
  const at::Tensor* weight = tensor(v[4], "weight");
  Call call(x, "x");
  const Rows rx(x, "x", call), rdy(dy, "dy", call);
  if (rdy.rows != rx.rows || rdy.cols != rx.cols) bad("dy must have x's shape");
  const at::Tensor* stat[2] = {&mean, &rstd};
  for (int i = 0; i < 2; i++)
    if (stat[i]->scalar_type() != at::kFloat || stat[i]->numel() != rx.rows || !stat[i]->is_contiguous() || !stat[i]->is_cuda() ||
        stat[i]->get_device() != x.get_device())
      bad(std::string(i ? "rstd" : "mean") + " must be " + std::to_string(rx.rows) + " contiguous float32 values on x's GPU");
  const at::ScalarType ptype = weight ? weight->scalar_type() : call.type;
  ringar_layer_norm_backward_t a = {};
  a.dtype = (ringar_dtype_t)call.code;
  a.param_dtype = (ringar_dtype_t)code_of(ptype);
  a.rows = rx.rows;
  a.cols = rx.cols;
  a.dy = rdy.p;
  a.lddy = rdy.ld;
  a.x = rx.p;
  a.ldx = rx.ld;
  a.mean = (const float*)mean.data_ptr();
  a.rstd = (const float*)rstd.data_ptr();
  a.weight = vec(weight, rx.cols, "weight", ptype, call);
  at::Tensor gx, gw, gb;
  if (truth(v[5], "dx")) gx = call.make(x.sizes());
  if (truth(v[6], "dweight")) gw = call.make({rx.cols}, ptype);
  if (truth(v[7], "dbias")) gb = call.make({rx.cols}, ptype);
  a.dx = ptr(gx);
  a.lddx = rx.cols;
  a.dweight = ptr(gw);
  a.dbias = ptr(gb);
  done(ringar_layer_norm_backward(&a, call.stream()), "ringar_layer_norm_backward");
  return tuple({wrap_or_none(gx), wrap_or_none(gw), wrap_or_none(gb)});
}

PyObject* forward(PyObject* const* v) {
  const at::Tensor &x = needed(v[0], "x"), &weight = needed(v[1], "weight");
  const at::Tensor *bias = tensor(v[2], "bias"), *residual = tensor(v[4], "residual"), *out = tensor(v[6], "out");
  const bool save_pre = truth(v[5], "save_pre"), gated = truth(v[7], "gated");
  Call call(x, "x");
  const Rows rx(x, "x", call), rw(weight, "weight", call);
  if (rw.cols != rx.cols || weight.dim() != 2 || (gated && rw.rows % 2))
    bad(gated ? "weight must be 2 out_features x in_features" : "weight must be out_features x in_features");
  const int64_t n = gated ? rw.rows / 2 : rw.rows;
  ringar_linear_t a = {};
  a.dtype = (ringar_dtype_t)call.code;
  a.act = (ringar_act_t)PyLong_AsLong(v[3]);
  a.rows = rx.rows;
  a.in_features = rx.cols;
  a.out_features = n;
  a.x = rx.p;
  a.ldx = rx.ld;
  a.weight = rw.p;
  a.ldw = rw.ld;
  a.bias = vec(bias, rw.rows, "bias", call.type, call);
  if (residual) {
    const Rows rr(*residual, "residual", call);
    if (rr.rows != rx.rows || rr.cols != n) bad("residual must have the output's shape");
    a.residual = rr.p;
    a.ldr = rr.ld;
  }
  const auto shape = shape_of(x, n);
  at::Tensor y, pre;
  if (out) {
    if (out->sizes() != at::IntArrayRef(shape)) bad("out must have shape x.shape[:-1] + (out_features,)");
    const Rows ry(*out, "out", call);
    y = *out;
    a.ldy = ry.ld;
  } else {
    y = call.make(shape);
    a.ldy = n;
  }
  a.y = y.data_ptr();
  if (save_pre) {
    pre = call.make(shape_of(x, rw.rows));
    a.pre = pre.data_ptr();
    a.ldp = rw.rows;
  }
  if (gated) done(ringar_gated_ffn(&a, call.stream()), "ringar_gated_ffn");
  else done(ringar_linear(&a, call.stream()), "ringar_linear");
  written(out);
  if (!save_pre) return wrap(y);
  return tuple({wrap(y), wrap(pre)});
}

PyObject* backward(PyObject* const* v) {
  const at::Tensor& dy = needed(v[0], "dy");
  const at::Tensor *x = tensor(v[1], "x"), *weight = tensor(v[2], "weight"), *pre = tensor(v[3], "pre");
  const bool want_x = truth(v[5], "dx"), want_w = truth(v[6], "dweight"), want_b = truth(v[7], "dbias"), gated = truth(v[8], "gated");
  Call call(dy, "dy");
  const Rows rdy(dy, "dy", call);
  const int64_t n = rdy.cols, wide = gated ? 2 * n : n;
  ringar_linear_backward_t a = {};
  a.dtype = (ringar_dtype_t)call.code;
  a.act = (ringar_act_t)PyLong_AsLong(v[4]);
  a.rows = rdy.rows;
  a.out_features = n;
  a.dy = rdy.p;
  a.lddy = rdy.ld;
  int64_t k = 0;
  if (x) {
    const Rows r(*x, "x", call);
    if (r.rows != rdy.rows) bad("x and dy must have the same rows");
    k = r.cols;
    a.x = r.p;
    a.ldx = r.ld;
  } else if (want_w) {
    bad("the weight's gradient needs x");
  }
  if (weight) {
    const Rows r(*weight, "weight", call);
    if (r.rows != wide || weight->dim() != 2 || (x && r.cols != k)) bad("weight does not fit dy and x");
    k = r.cols;
    a.weight = r.p;
    a.ldw = r.ld;
  } else if (want_x) {
    bad("x's gradient needs the weight");
  }
  a.in_features = k;
  if (pre) {
    const Rows r(*pre, "pre", call);
    if (r.rows != rdy.rows || r.cols != wide) bad("pre must have " + std::to_string(wide) + " columns and dy's rows");
    a.pre = r.p;
    a.ldp = r.ld;
  } else if (gated || a.act != RINGAR_ACT_NONE) {
    bad("pre, kept by the forward pass, is needed");
  }
  at::Tensor gx, gw, gb;
  if (want_x) gx = call.make(shape_of(dy, k));
  if (want_w) gw = call.make({wide, k});
  if (want_b) gb = call.make({wide});
  a.dx = ptr(gx);
  a.lddx = a.lddw = k;
  a.dweight = ptr(gw);
  a.dbias = ptr(gb);
  if (gated) done(ringar_gated_ffn_backward(&a, call.stream()), "ringar_gated_ffn_backward");
  else done(ringar_linear_backward(&a, call.stream()), "ringar_linear_backward");
  return tuple({wrap_or_none(gx), wrap_or_none(gw), wrap_or_none(gb)});
}

PyObject* raise(const Refusal& r) {
  PyObject* m = PyImport_ImportModule("ring_allreduce_reduce_amd");
  PyObject* cls = m ? PyObject_GetAttrString(m, "RingarError") : nullptr;
  PyObject* e = cls ? PyObject_CallFunction(cls, "is", r.code, r.what.c_str()) : nullptr;
  if (e) PyErr_SetObject(cls, e);
  Py_XDECREF(e);
  Py_XDECREF(cls);
  Py_XDECREF(m);
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N> PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refusal& r) {
    return raise(r);
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N> PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)(void))(PyObject * (*)(PyObject*, PyObject* const*, Py_ssize_t)) entry<F, N>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<layer_norm, 6>("layer_norm"),
    method<layer_norm_backward, 8>("layer_norm_backward"),
    method<forward, 8>("forward"),
    method<backward, 9>("backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_ext() { return PyModule_Create(&module); }
