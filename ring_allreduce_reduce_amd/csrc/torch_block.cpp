// The block operators on torch tensors: argument checks, output tensors and
// the C call, in one extension function each (a call of a few microseconds
// spends most of them here; the same checks in Python took 4 us more).
// Signatures, defaults and streams are block.py's.
#include "torch_args.h"

using namespace ringar_torch;

namespace {

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
    method<rms_norm, 8>("rms_norm"),
    method<rms_norm_backward, 7>("rms_norm_backward"),
    method<dropout, 8>("dropout"),
    method<cross_attention, 7>("cross_attention"),
    method<cross_attention_backward, 11>("cross_attention_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_ext() { return PyModule_Create(&module); }
