// The root-mean-square norm, dropout and cross attention on torch tensors:
// argument checks, output tensors and the C call, one extension function each.
// Signatures, defaults and streams are block.py's and attention.py's.
#include "torch_args.h"

namespace ringar_torch {

namespace {

// A number, or a Python error.
bool number(PyObject* o, double* to) {
  *to = PyFloat_AsDouble(o);
  return !(*to == -1.0 && PyErr_Occurred());
}

int64_t whole(PyObject* o, const char* what) {
  if (!PyLong_Check(o)) bad(std::string(what) + " must be a whole number");
  const int64_t n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(std::string(what) + " is out of range");
  }
  return n;
}

uint64_t word(PyObject* o, const char* what) {
  if (!PyLong_Check(o)) bad(std::string(what) + " must be a whole number");
  const uint64_t n = PyLong_AsUnsignedLongLong(o);
  if (n == (uint64_t)-1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(std::string(what) + " must lie in 0 .. 2^64 - 1");
  }
  return n;
}

// float32 statistics of `n` rows
const float* stats_of(const at::Tensor& t, int64_t n, const char* what, const Call& call) {
  if (t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous() || !t.is_cuda() || t.get_device() != call.of.get_device())
    bad(std::string(what) + " must be " + std::to_string(n) + " contiguous float32 values on the operands' GPU");
  return (const float*)t.data_ptr();
}

// Rows of `t` where it has the shape of `like`.
Rows like_rows(const at::Tensor& t, const at::Tensor& like, const char* what, const char* as, const Call& call) {
  if (t.sizes() != like.sizes()) bad(std::string(what) + " must have " + as + "'s shape");
  return Rows(t, what, call);
}

struct Heads {
  void* p;
  int64_t batch, rows, heads, dim;
  int64_t strides[3];

  Heads(const at::Tensor& t, const char* what, const Call& call) {
    if (t.scalar_type() != call.type || !t.is_cuda() || t.get_device() != call.of.get_device())
      bad(std::string(what) + " must have the dtype and device of the other operands");
    if (t.dim() != 4) bad(std::string(what) + " must have the dimensions (batch, rows, heads, head_dim)");
    if (t.size(3) > 1 && t.stride(3) != 1) bad(std::string(what) + ": the last dimension must be contiguous");
    p = t.data_ptr();
    batch = t.size(0);
    rows = t.size(1);
    heads = t.size(2);
    dim = t.size(3);
    for (int i = 0; i < 3; i++) strides[i] = t.stride(i);
  }
  void to(const void** at, int64_t* s) const {
    *at = p;
    for (int i = 0; i < 3; i++) s[i] = strides[i];
  }
};

const int32_t* lengths_of(const at::Tensor* t, int64_t batch, const Call& call) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != batch || !t->is_contiguous() || !t->is_cuda() ||
      t->get_device() != call.of.get_device())
    bad("key_lengths must be a contiguous vector of " + std::to_string(batch) + " int32 values on the operands' GPU");
  return (const int32_t*)t->data_ptr();
}

// The sizes that q, k and v give; scale: 1 / sqrt(head_dim) by default.
template <typename A> bool sizes(A& a, const Call& call, const Heads& q, const Heads& k, const Heads& v, PyObject* scale) {
  if (k.batch != q.batch || k.dim != q.dim) bad("k must have q's batch and head_dim");
  if (v.batch != k.batch || v.rows != k.rows || v.heads != k.heads || v.dim != k.dim) bad("v must have k's shape");
  a.dtype = (ringar_dtype_t)call.code;
  a.batch = q.batch;
  a.queries = q.rows;
  a.keys = k.rows;
  a.heads = q.heads;
  a.kv_heads = k.heads;
  a.head_dim = q.dim;
  q.to(&a.q, a.q_strides);
  k.to(&a.k, a.k_strides);
  v.to(&a.v, a.v_strides);
  double s = 1.0 / std::sqrt((double)(q.dim > 0 ? q.dim : 1));
  if (scale != Py_None && !number(scale, &s)) return false;
  a.scale = (float)s;
  return true;
}

}  // namespace

PyObject* rms_norm(PyObject* const* v) {
  const at::Tensor& x = needed(v[0], "x");
  const at::Tensor *weight = tensor(v[1], "weight"), *residual = tensor(v[3], "residual"), *out = tensor(v[6], "out"),
                   *sum_out = tensor(v[7], "sum_out");
  double eps;
  if (!number(v[2], &eps)) return nullptr;
  const int kind = (int)PyLong_AsLong(v[4]);
  const bool stats = truth(v[5], "stats");
  Call call(x, "x");
  const Rows rx(x, "x", call);
  const at::ScalarType ptype = weight ? weight->scalar_type() : call.type;
  ringar_rms_norm_t a = {};
  a.dtype = (ringar_dtype_t)call.code;
  a.param_dtype = (ringar_dtype_t)code_of(ptype);
  a.out = (ringar_out_t)kind;
  a.rows = rx.rows;
  a.cols = rx.cols;
  a.x = rx.p;
  a.ldx = rx.ld;
  a.weight = vec(weight, rx.cols, "weight", ptype, call);
  a.eps = (float)eps;
  at::Tensor y, scale, sum, rstd;
  if (residual) {
    const Rows rr = like_rows(*residual, x, "residual", "x", call);
    a.residual = rr.p;
    a.ldr = rr.ld;
    if (sum_out) {
      const Rows rs = like_rows(*sum_out, x, "sum_out", "x", call);
      sum = *sum_out;
      a.lds = rs.ld;
    } else {
      sum = call.make(x.sizes());
      a.lds = rx.cols;
    }
    a.sum = sum.data_ptr();
  } else if (sum_out) {
    bad("sum_out needs a residual");
  }
  if (kind != RINGAR_OUT_SAME) {
    y = call.make(x.sizes(), at::kFloat8_e4m3fn);
    scale = call.make(shape_of(x, kind == RINGAR_OUT_FP8_ROW ? 1 : (rx.cols + 127) / 128), at::kFloat);
    a.scale = (float*)scale.data_ptr();
    a.ldy = rx.cols;
  } else if (out) {
    const Rows ry = like_rows(*out, x, "out", "x", call);
    y = *out;
    a.ldy = ry.ld;
  } else {
    y = call.make(x.sizes());
    a.ldy = rx.cols;
  }
  a.y = y.data_ptr();
  if (stats) {
    rstd = call.make(x.sizes().slice(0, x.dim() - 1), at::kFloat);
    a.rstd = (float*)rstd.data_ptr();
  }
  done(ringar_rms_norm(&a, call.stream()), "ringar_rms_norm");
  written(out);
  written(sum_out);
  if (!scale.defined() && !sum.defined() && !stats) return wrap(y);
  PyObject* r = PyTuple_New(1 + scale.defined() + sum.defined() + rstd.defined());
  Py_ssize_t i = 0;
  for (at::Tensor* t : {&y, &scale, &sum, &rstd})
    if (t->defined()) PyTuple_SET_ITEM(r, i++, wrap(*t));
  return r;
}

PyObject* rms_norm_backward(PyObject* const* v) {
  const at::Tensor &dy = needed(v[0], "dy"), &x = needed(v[1], "x"), &rstd = needed(v[2], "rstd");
  const at::Tensor *weight = tensor(v[3], "weight"), *dsum = tensor(v[4], "dsum");
  Call call(x, "x");
  const Rows rx(x, "x", call), rdy = like_rows(dy, x, "dy", "x", call);
  const at::ScalarType ptype = weight ? weight->scalar_type() : call.type;
  ringar_rms_norm_backward_t a = {};
  a.dtype = (ringar_dtype_t)call.code;
  a.param_dtype = (ringar_dtype_t)code_of(ptype);
  a.rows = rx.rows;
  a.cols = rx.cols;
  a.dy = rdy.p;
  a.lddy = rdy.ld;
  a.x = rx.p;
  a.ldx = rx.ld;
  a.rstd = stats_of(rstd, rx.rows, "rstd", call);
  a.weight = vec(weight, rx.cols, "weight", ptype, call);
  if (dsum) {
    const Rows rs = like_rows(*dsum, x, "dsum", "x", call);
    a.dsum = rs.p;
    a.ldds = rs.ld;
  }
  at::Tensor gx, gw;
  if (truth(v[5], "dx")) gx = call.make(x.sizes());
  if (truth(v[6], "dweight")) gw = call.make({rx.cols}, ptype);
  a.dx = ptr(gx);
  a.lddx = rx.cols;
  a.dweight = ptr(gw);
  done(ringar_rms_norm_backward(&a, call.stream()), "ringar_rms_norm_backward");
  return tuple({wrap_or_none(gx), wrap_or_none(gw)});
}

PyObject* dropout(PyObject* const* v) {
  const at::Tensor& x = needed(v[0], "x");
  const at::Tensor *residual = tensor(v[4], "residual"), *out = tensor(v[7], "out");
  ringar_dropout_t a = {};
  if (!number(v[1], &a.p)) return nullptr;
  a.seed = word(v[2], "seed");
  const at::Tensor* more = THPVariable_Check(v[3]) ? tensor(v[3], "offset") : nullptr;
  Call call(x, "x");
  if (more) {
    if (more->scalar_type() != at::kLong || more->numel() != 1 || !more->is_cuda() || more->get_device() != x.get_device())
      bad("an offset in memory must be one int64 value on x's GPU");
    a.more_offset = (const int64_t*)more->data_ptr();
  } else {
    a.offset = word(v[3], "offset");
  }
  a.first_row = whole(v[5], "first_row");
  a.first_col = whole(v[6], "first_col");
  const Rows rx(x, "x", call);
  a.dtype = (ringar_dtype_t)call.code;
  a.rows = rx.rows;
  a.cols = rx.cols;
  a.x = rx.p;
  a.ldx = rx.ld;
  if (residual) {
    const Rows rr = like_rows(*residual, x, "residual", "x", call);
    a.residual = rr.p;
    a.ldr = rr.ld;
  }
  at::Tensor y;
  if (out) {
    const Rows ry = like_rows(*out, x, "out", "x", call);
    y = *out;
    a.ldy = ry.ld;
  } else {
    y = call.make(x.sizes());
    a.ldy = rx.cols;
  }
  a.y = y.data_ptr();
  done(ringar_dropout(&a, call.stream()), "ringar_dropout");
  written(out);
  return wrap(y);
}

PyObject* cross_attention(PyObject* const* v) {
  const at::Tensor &q = needed(v[0], "q"), &k = needed(v[1], "k"), &val = needed(v[2], "v");
  const at::Tensor *lengths = tensor(v[3], "key_lengths"), *out = tensor(v[6], "out");
  const bool stats = truth(v[5], "stats");
  Call call(q, "q");
  const Heads hq(q, "q", call), hk(k, "k", call), hv(val, "v", call);
  ringar_cross_attention_t a = {};
  if (!sizes(a, call, hq, hk, hv, v[4])) return nullptr;
  a.key_lengths = lengths_of(lengths, hq.batch, call);
  at::Tensor y, lse;
  if (out) {
    if (out->sizes() != q.sizes()) bad("out must have q's shape");
    y = *out;
  } else {
    y = call.make(q.sizes());
  }
  const Heads hy(y, "out", call);
  a.y = hy.p;
  for (int i = 0; i < 3; i++) a.y_strides[i] = hy.strides[i];
  if (stats) {
    lse = call.make({hq.batch, hq.heads, hq.rows}, at::kFloat);
    a.lse = (float*)lse.data_ptr();
  }
  done(ringar_cross_attention(&a, call.stream()), "ringar_cross_attention");
  written(out);
  if (!stats) return wrap(y);
  return tuple({wrap(y), wrap(lse)});
}

PyObject* cross_attention_backward(PyObject* const* v) {
  const at::Tensor &dy = needed(v[0], "dy"), &q = needed(v[1], "q"), &k = needed(v[2], "k"), &val = needed(v[3], "v"), &y = needed(v[4], "y"),
                   &lse = needed(v[5], "lse");
  const at::Tensor* lengths = tensor(v[6], "key_lengths");
  Call call(q, "q");
  const Heads hq(q, "q", call), hk(k, "k", call), hv(val, "v", call), hdy(dy, "dy", call), hy(y, "y", call);
  if (dy.sizes() != q.sizes() || y.sizes() != q.sizes()) bad("dy and y must have q's shape");
  ringar_cross_attention_backward_t a = {};
  if (!sizes(a, call, hq, hk, hv, v[7])) return nullptr;
  hdy.to(&a.dy, a.dy_strides);
  hy.to(&a.y, a.y_strides);
  a.lse = stats_of(lse, hq.batch * hq.heads * hq.rows, "lse", call);
  a.key_lengths = lengths_of(lengths, hq.batch, call);
  at::Tensor gq, gk, gv;
  if (truth(v[8], "dq")) gq = call.make(q.sizes());
  if (truth(v[9], "dk")) gk = call.make(k.sizes());
  if (truth(v[10], "dv")) gv = call.make(val.sizes());
  a.dq = ptr(gq);
  a.dk = ptr(gk);
  a.dv = ptr(gv);
  done(ringar_cross_attention_backward(&a, call.stream()), "ringar_cross_attention_backward");
  return tuple({wrap_or_none(gq), wrap_or_none(gk), wrap_or_none(gv)});
}

}  // namespace ringar_torch
