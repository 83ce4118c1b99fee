// C ABI of the block operators: argument checks, workspaces and launches of
// layer norm, the linear product with its epilogue, and the gated
// feed-forward, each with its backward pass.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <tuple>
#include <vector>

#include "block_types.h"
#include "op_checks.h"
#include "ringar.h"

using namespace ringar;

namespace {

// ------------------------------------------------------------- workspaces
// One buffer per (device, stream), grown as calls need it and reused in
// stream order.  The mutex is held from asking for the buffer to the last
// launch that uses it, so two threads on one stream cannot interleave.
struct Workspace {
  int device = 0;
  char* p = nullptr;
  size_t bytes = 0;
  bool captured_ever = false;          // a graph may hold this buffer's address
  std::vector<void*> retired;          // replaced buffers such graphs may hold
};

// hipStreamPerThread is one handle for a stream of every host thread: there
// the thread's number (never used again) tells the streams apart.
uint64_t thread_of(hipStream_t st) {
  static std::atomic<uint64_t> threads{0};
  if (st != hipStreamPerThread) return 0;
  static thread_local const uint64_t mine = ++threads;
  return mine;
}

std::map<std::tuple<int, hipStream_t, uint64_t>, Workspace> g_ws;

// ---------------------------------------------------------------- checks
// Null where something is to be read or written, misalignment, a row stride
// below the row's length (inputs may repeat one row: stride 0).
ringar_result_t check_mat(const Mat& m) {
  if (m.rows == 0 || m.cols == 0) return RINGAR_SUCCESS;
  if (!m.p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, std::string(m.name) + " is null");
  if ((uintptr_t)m.p % m.es) return refuse(RINGAR_ERR_INVALID_ARGUMENT, std::string(m.name) + " is not aligned to its element size");
  if (m.rows > 1 && m.ld < m.cols && !(m.ld == 0 && !m.output))
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, std::string(m.name) + ": row stride below the row's length");
  if (m.ld > kMaxPitch) return refuse(RINGAR_ERR_INVALID_ARGUMENT, std::string(m.name) + ": row stride beyond 2^31 - 1 elements");
  return RINGAR_SUCCESS;
}

bool overlap(const Mat& a, const Mat& b) {
  if (!a.p || !b.p || !a.rows || !b.rows || !a.cols || !b.cols) return false;
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  const uintptr_t ea = pa + ((uint64_t)(a.rows - 1) * a.ld + a.cols) * a.es;
  const uintptr_t eb = pb + ((uint64_t)(b.rows - 1) * b.ld + b.cols) * b.es;
  if (pa >= eb || pb >= ea) return false;
  // columns of one array: same row stride (a single row goes by the other's),
  // column ranges apart
  const uint64_t pitch_a = a.rows > 1 ? (uint64_t)a.ld * a.es : 0, pitch_b = b.rows > 1 ? (uint64_t)b.ld * b.es : 0;
  const uint64_t pitch = pitch_a ? pitch_a : pitch_b;
  if (pitch && (a.rows == 1 || pitch_a == pitch) && (b.rows == 1 || pitch_b == pitch)) {
    const uint64_t d = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;
    if (d >= a.cols * a.es && d + b.cols * b.es <= pitch) return false;
  }
  return true;
}

bool same_place(const Mat& a, const Mat& b) { return a.p == b.p && (a.ld == b.ld || a.rows <= 1) && a.es == b.es; }

}  // namespace

namespace ringar {

std::mutex g_ws_mu;

// The call's result tells of the error: nothing of it is left for
// hipGetLastError().
ringar_result_t hip_fail(hipError_t e, const char* what) {
  (void)hipGetLastError();
  last_error_text() = std::string(what) + ": " + hipGetErrorString(e);
  return RINGAR_ERR_DEVICE;
}

ringar_result_t refuse(ringar_result_t code, const std::string& why) {
  last_error_text() = why;
  return code;
}

ringar_result_t workspace(hipStream_t st, size_t bytes, char** out) {
  *out = nullptr;
  if (bytes == 0) return RINGAR_SUCCESS;
  bytes += kCounterBytes;
  int dev = 0;
  HIP_TRY(hipGetDevice(&dev));
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  HIP_TRY(hipStreamIsCapturing(st, &cap));
  Workspace& w = g_ws[std::make_tuple(dev, st, thread_of(st))];
  w.device = dev;
  if (cap != hipStreamCaptureStatusNone) {
    if (w.bytes < bytes)
      return refuse(RINGAR_ERR_INVALID_USAGE,
                    "stream capture: the stream must have run a call of this shape first (its workspace is not allocated)");
    w.captured_ever = true;
  } else if (w.bytes < bytes) {
    HIP_TRY(hipStreamSynchronize(st));
    if (w.p && w.captured_ever) w.retired.push_back(w.p);
    else if (w.p) HIP_TRY(hipFree(w.p));
    w.p = nullptr;
    w.bytes = 0;
    w.captured_ever = false;
    const size_t want = (bytes + (4u << 20) - 1) / (4u << 20) * (4u << 20);
    HIP_TRY(hipMalloc((void**)&w.p, want));
    const hipError_t e = launch_clear((uint32_t*)w.p, kCounters, st);
    if (e != hipSuccess) {                   // counters unset: the next call starts over
      (void)hipFree(w.p);
      w.p = nullptr;
      return hip_fail(e, "clearing the workspace's counters");
    }
    w.bytes = want;
  }
  *out = w.p + kCounterBytes;
  return RINGAR_SUCCESS;
}

// Every operand's own checks, and no output over another operand.  The one
// exception is an operand marked `in_place` or `any_place` (its elements are read
// before the output's are written, by the same thread); another one that lies at the
// same address, say a square product's x that is the residual too, is refused.
ringar_result_t check_mats(std::initializer_list<Mat> all) {
  for (const Mat& m : all) TRY(check_mat(m));
  for (const Mat* o = all.begin(); o != all.end(); o++) {
    if (!o->output) continue;
    for (const Mat* m = all.begin(); m != all.end(); m++) {
      if (m == o || (m->output && m < o)) continue;
      if ((m->any_place || (m->in_place && !strcmp(o->name, "y"))) && same_place(*m, *o)) continue;
      if (overlap(*o, *m))
        return refuse(RINGAR_ERR_INVALID_USAGE, std::string(o->name) + " overlaps " + m->name);
    }
  }
  return RINGAR_SUCCESS;
}

}  // namespace ringar

namespace {

// --------------------------------------------------------------- products
// `ws`: p.bytes at `at` in the stream's workspace (null where nothing of it
// is needed).
ringar_result_t run_gemm(int dtype, const GemmPlan& p, char* ws, size_t at, hipStream_t st) {
  HIP_TRY(launch_gemm(dtype, p, ws ? ws + at : nullptr, ws ? (uint32_t*)(ws - kCounterBytes) : nullptr, st));
  return RINGAR_SUCCESS;
}

ringar_result_t check_plan(const GemmPlan& p) {
  if (p.too_many) return refuse(RINGAR_ERR_INVALID_USAGE, "the product has more tiles than one launch takes");
  return RINGAR_SUCCESS;
}

}  // namespace

namespace ringar {

bool release_workspaces() {
  std::lock_guard<std::mutex> lock(g_ws_mu);
  auto go = [](hipError_t e, const char* what) {
    if (e == hipSuccess) return true;
    hip_fail(e, what);
    return false;
  };
  int cur = 0;
  if (!go(hipGetDevice(&cur), "hipGetDevice")) return false;
  for (auto& kv : g_ws) {
    Workspace& w = kv.second;
    if (!go(hipSetDevice(w.device), "hipSetDevice") || !go(hipDeviceSynchronize(), "hipDeviceSynchronize")) return false;
    if (w.p && !go(hipFree(w.p), "hipFree")) return false;
    w.p = nullptr;
    w.bytes = 0;
    for (void* p : w.retired)
      if (!go(hipFree(p), "hipFree")) return false;
    w.retired.clear();
  }
  g_ws.clear();
  return go(hipSetDevice(cur), "hipSetDevice");
}

}  // namespace ringar

static ringar_result_t norm_forward(const ringar_layer_norm_t* p, ringar_stream_t stream) {
  if (!p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "null arguments");
  if (!type_ok(p->dtype) || (p->param_dtype != p->dtype && p->param_dtype != RINGAR_FLOAT32))
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "layer norm takes fp16, bf16 or fp32, its parameters in the same type or fp32");
  if (!dims_ok({p->rows, p->cols}) || p->cols == 0) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "rows or cols out of range");
  if (!(p->eps >= 0.0f)) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "eps below zero");
  const size_t es = size_of(p->dtype), ws = size_of(p->param_dtype);
  TRY(check_mats({{"x", p->x, p->rows, p->cols, p->ldx, es, false, true},
                  VEC("weight", p->weight, p->cols, ws, false),
                  VEC("bias", p->bias, p->cols, ws, false),
                  {"y", p->y, p->rows, p->cols, p->ldy, es, true},
                  VEC("mean", p->mean, p->rows, 4, true),
                  VEC("rstd", p->rstd, p->rows, 4, true)}));
  if (p->rows == 0) return RINGAR_SUCCESS;
  NormArgs a = {};
  a.x = p->x;
  a.weight = p->weight;
  a.bias = p->bias;
  a.y = p->y;
  a.mean = p->mean;
  a.rstd = p->rstd;
  a.ldx = p->ldx;
  a.ldy = p->ldy;
  a.rows = p->rows;
  a.cols = (int)p->cols;
  a.eps = p->eps;
  a.inv_cols = 1.0f / (float)p->cols;
  HIP_TRY(launch_norm_forward(p->dtype, p->param_dtype, a, (hipStream_t)stream));
  return RINGAR_SUCCESS;
}

static ringar_result_t norm_backward(const ringar_layer_norm_backward_t* p, ringar_stream_t stream) {
  if (!p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "null arguments");
  if (!type_ok(p->dtype) || (p->param_dtype != p->dtype && p->param_dtype != RINGAR_FLOAT32))
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "layer norm takes fp16, bf16 or fp32, its parameters in the same type or fp32");
  if (!dims_ok({p->rows, p->cols}) || p->cols == 0) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "rows or cols out of range");
  const size_t es = size_of(p->dtype), ws = size_of(p->param_dtype);
  TRY(check_mats({{"dy", p->dy, p->rows, p->cols, p->lddy, es, false},
                  {"x", p->x, p->rows, p->cols, p->ldx, es, false},
                  {"mean", p->mean, 1, p->rows, p->rows, 4, false},
                  {"rstd", p->rstd, 1, p->rows, p->rows, 4, false},
                  VEC("weight", p->weight, p->cols, ws, false),
                  {"dx", p->dx, p->dx ? p->rows : 0, p->cols, p->lddx, es, true},
                  VEC("dweight", p->dweight, p->cols, ws, true),
                  VEC("dbias", p->dbias, p->cols, ws, true)}));
  const bool params = p->dweight || p->dbias;
  if (!params && (!p->dx || p->rows == 0)) return RINGAR_SUCCESS;
  hipStream_t st = (hipStream_t)stream;
  NormArgs a = {};
  a.x = p->x;
  a.dy = p->dy;
  a.weight = p->weight;
  a.y = p->dx;
  a.mean = (float*)p->mean;
  a.rstd = (float*)p->rstd;
  a.ldx = p->ldx;
  a.lddy = p->lddy;
  a.ldy = p->lddx;
  a.rows = p->rows;
  a.cols = (int)p->cols;
  a.inv_cols = 1.0f / (float)p->cols;
  a.groups = norm_backward_groups(p->rows, a.cols);
  std::lock_guard<std::mutex> lock(g_ws_mu);
  const bool split = params && (a.groups != 1 || p->cols > kNormLongest);
  if (split) {
    char* ws_p = nullptr;
    TRY(workspace(st, (size_t)2 * a.groups * p->cols * 4, &ws_p));
    a.part = (float*)ws_p;
  } else {
    a.dweight = p->dweight;
    a.dbias = p->dbias;
  }
  if (p->rows) HIP_TRY(launch_norm_backward(p->dtype, p->param_dtype, a, st));
  if (split)
    HIP_TRY(launch_col_sum(p->param_dtype, {a.part, a.groups, 2 * p->cols, p->cols, p->dweight, p->dbias}, st));
  return RINGAR_SUCCESS;
}

static ringar_result_t product_forward(const ringar_linear_t* p, bool gated, hipStream_t st) {
  if (!p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "null arguments");
  if (!type_ok(p->dtype)) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "products take fp16, bf16 or fp32");
  if (p->act < RINGAR_ACT_NONE || p->act > RINGAR_ACT_SIGMOID) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "unknown activation");
  const int64_t wide = gated ? 2 * p->out_features : p->out_features;
  if (!dims_ok({p->rows, p->in_features, p->out_features, wide})) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "a size is out of range");
  if (gated && p->residual) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "the gated feed-forward takes no residual");
  const size_t es = size_of(p->dtype);
  TRY(check_mats({{"x", p->x, p->rows, p->in_features, p->ldx, es, false},
                  {"weight", p->weight, wide, p->in_features, p->ldw, es, false},
                  VEC("bias", p->bias, wide, es, false),
                  {"residual", p->residual, p->residual ? p->rows : 0, p->out_features, p->ldr, es, false, true},
                  {"y", p->y, p->rows, p->out_features, p->ldy, es, true},
                  {"pre", p->pre, p->pre ? p->rows : 0, wide, p->ldp, es, true}}));
  if (p->rows == 0 || p->out_features == 0) return RINGAR_SUCCESS;
  const int epi = gated ? kEpiGated : kEpiLinear;
  GemmArgs a = {};
  a.a = p->x;
  a.b = p->weight;
  a.sam = p->ldx;
  a.sbn = p->ldw;
  a.sak = a.sbk = 1;
  a.m = (int)p->rows;
  a.n = (int)p->out_features;
  a.k = (int)p->in_features;
  a.bias = p->bias;
  a.residual = p->residual;
  a.c = p->y;
  a.pre = p->pre;
  a.ldc = p->ldy;
  a.ldr = p->ldr;
  a.ldp = p->ldp;
  a.act = p->act;
  const GemmPlan plan = plan_gemm(p->dtype, epi, a);
  TRY(check_plan(plan));
  std::lock_guard<std::mutex> lock(g_ws_mu);
  char* ws = nullptr;
  TRY(workspace(st, plan.bytes, &ws));
  return run_gemm(p->dtype, plan, ws, 0, st);
}

static ringar_result_t product_backward(const ringar_linear_backward_t* p, bool gated, hipStream_t st) {
  if (!p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "null arguments");
  if (!type_ok(p->dtype)) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "products take fp16, bf16 or fp32");
  if (p->act < RINGAR_ACT_NONE || p->act > RINGAR_ACT_SIGMOID) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "unknown activation");
  const int64_t wide = gated ? 2 * p->out_features : p->out_features;
  if (!dims_ok({p->rows, p->in_features, p->out_features, wide})) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "a size is out of range");
  const bool use_pre = gated || p->act != RINGAR_ACT_NONE;
  const size_t es = size_of(p->dtype);
  TRY(check_mats({{"dy", p->dy, p->rows, p->out_features, p->lddy, es, false},
                  {"pre", use_pre ? p->pre : nullptr, use_pre ? p->rows : 0, wide, p->ldp, es, false},
                  {"x", p->x, p->dweight ? p->rows : 0, p->in_features, p->ldx, es, false},
                  {"weight", p->weight, p->dx ? wide : 0, p->in_features, p->ldw, es, false},
                  {"dx", p->dx, p->dx ? p->rows : 0, p->in_features, p->lddx, es, true},
                  {"dweight", p->dweight, p->dweight ? wide : 0, p->in_features, p->lddw, es, true},
                  VEC("dbias", p->dbias, wide, es, true)}));
  if (few_rows(p->dtype, p->rows, wide, p->in_features)) {
    if (!p->dx && !p->dweight && !p->dbias) return RINGAR_SUCCESS;
    FewArgs f = {};
    f.dy = p->dy;
    f.pre = use_pre ? p->pre : nullptr;
    f.x = p->x;
    f.w = p->weight;
    f.dx = p->dx;
    f.dw = p->dweight;
    f.db = p->dbias;
    f.lddy = p->lddy;
    f.ldp = p->ldp;
    f.ldx = p->ldx;
    f.ldw = p->ldw;
    f.lddx = p->lddx;
    f.lddw = p->lddw;
    f.k = p->in_features;
    f.rows = (int)p->rows;
    f.n = (int)p->out_features;
    f.wide = (int)wide;
    f.act = p->act;
    f.gated = gated;
    const size_t part = plan_few(p->dtype, f);
    std::lock_guard<std::mutex> lock(g_ws_mu);
    char* ws = nullptr;
    TRY(workspace(st, part, &ws));
    f.part = (float*)ws;
    HIP_TRY(launch_few(p->dtype, f, st));
    return RINGAR_SUCCESS;
  }
  // dz = dy where there is nothing to undo
  const bool need_dz = use_pre && (p->dx || p->dweight);
  DzArgs z = {};
  z.dy = p->dy;
  z.pre = use_pre ? p->pre : nullptr;
  z.lddy = p->lddy;
  z.ldp = p->ldp;
  z.lddz = (wide + 63) / 64 * 64;
  z.rows = p->rows;
  z.n = (int)p->out_features;
  z.groups = p->rows && p->out_features ? dz_groups(p->dtype, p->rows, p->out_features) : 0;
  z.act = p->act;
  z.gated = gated;
  // dx[m][k] = sum_n dz[m][n] w[n][k];  dw[n][k] = sum_m dz[m][n] x[m][k]
  GemmArgs gx = {}, gw = {};
  gx.b = p->weight;
  gx.sak = 1;
  gx.sbn = 1;
  gx.sbk = p->ldw;
  gx.m = (int)p->rows;
  gx.n = (int)p->in_features;
  gx.k = (int)wide;
  gx.c = p->dx;
  gx.ldc = p->lddx;
  gw.b = p->x;
  gw.sam = 1;
  gw.sbn = 1;
  gw.sbk = p->ldx;
  gw.m = (int)wide;
  gw.n = (int)p->in_features;
  gw.k = (int)p->rows;
  gw.c = p->dweight;
  gw.ldc = p->lddw;
  // a workspace starts at a 256-byte boundary, like this stand-in for it
  gx.a = gw.a = need_dz ? (const void*)256 : p->dy;
  gx.sam = gw.sak = need_dz ? z.lddz : p->lddy;
  GemmPlan px = {}, pw = {};
  const bool together = p->dx && p->dweight && plan_gradients(p->dtype, gx, gw, &px, &pw);
  if (p->dx && !p->dweight) px = plan_gemm(p->dtype, kEpiStore, gx);
  if (p->dweight && !p->dx) pw = plan_gemm(p->dtype, kEpiStore, gw);
  TRY(check_plan(px));
  TRY(check_plan(pw));
  Layout l;
  const size_t at_dz = l.add(need_dz ? (size_t)p->rows * z.lddz * es : 0);
  const size_t at_sum = l.add(p->dbias ? (size_t)z.groups * wide * 4 : 0);
  const size_t at_x = l.add(together ? px.bytes : px.bytes > pw.bytes ? px.bytes : pw.bytes);
  const size_t at_w = together ? l.add(pw.bytes) : at_x;
  std::lock_guard<std::mutex> lock(g_ws_mu);
  char* ws = nullptr;
  TRY(workspace(st, l.bytes, &ws));
  if (need_dz) px.args.a = pw.args.a = z.dz = ws + at_dz;
  if (p->dbias && z.groups == 1) z.sums = p->dbias;
  else if (p->dbias && z.groups) z.part = (float*)(ws + at_sum);
  if ((z.dz || z.part || z.sums) && z.groups) HIP_TRY(launch_dz(p->dtype, z, st));
  // the bias's parts (none: zeros), beside the products or in a launch of their own
  const ColSumArgs sums = {z.part, z.groups, p->dbias && !z.sums ? wide : 0, wide, p->dbias, nullptr};
  if (sums.width && !together) HIP_TRY(launch_col_sum(p->dtype, sums, st));
  if (together) {
    HIP_TRY(launch_gradients(p->dtype, px, pw, sums, ws ? ws + at_x : nullptr, ws ? ws + at_w : nullptr, st));
  } else {
    if (p->dx) TRY(run_gemm(p->dtype, px, ws, at_x, st));
    if (p->dweight) TRY(run_gemm(p->dtype, pw, ws, at_w, st));
  }
  return RINGAR_SUCCESS;
}

extern "C" {

ringar_result_t ringar_layer_norm(const ringar_layer_norm_t* args, ringar_stream_t stream) {
  return guarded([&] { return norm_forward(args, stream); });
}

ringar_result_t ringar_layer_norm_backward(const ringar_layer_norm_backward_t* args, ringar_stream_t stream) {
  return guarded([&] { return norm_backward(args, stream); });
}

ringar_result_t ringar_linear(const ringar_linear_t* args, ringar_stream_t stream) {
  return guarded([&] { return product_forward(args, false, (hipStream_t)stream); });
}

ringar_result_t ringar_gated_ffn(const ringar_linear_t* args, ringar_stream_t stream) {
  return guarded([&] { return product_forward(args, true, (hipStream_t)stream); });
}

ringar_result_t ringar_linear_backward(const ringar_linear_backward_t* args, ringar_stream_t stream) {
  return guarded([&] { return product_backward(args, false, (hipStream_t)stream); });
}

ringar_result_t ringar_gated_ffn_backward(const ringar_linear_backward_t* args, ringar_stream_t stream) {
  return guarded([&] { return product_backward(args, true, (hipStream_t)stream); });
}

}  // extern "C"
