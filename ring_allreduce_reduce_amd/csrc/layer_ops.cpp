// C ABI of the root-mean-square norm and of dropout: argument checks and
// launches.
#include <cmath>

#include "layer_types.h"
#include "op_checks.h"

using namespace ringar;

static ringar_result_t check_rms(int dtype, int param_dtype, int64_t rows, int64_t cols) {
  if (!type_ok(dtype) || (param_dtype != dtype && param_dtype != RINGAR_FLOAT32))
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "the norm takes fp16, bf16 or fp32, its weight in the same type or fp32");
  if (!dims_ok({rows, cols}) || cols == 0) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "rows or cols out of range");
  return RINGAR_SUCCESS;
}

static ringar_result_t rms_forward(const ringar_rms_norm_t* p, ringar_stream_t stream) {
  if (!p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "null arguments");
  TRY(check_rms(p->dtype, p->param_dtype, p->rows, p->cols));
  if (p->out < RINGAR_OUT_SAME || p->out > RINGAR_OUT_FP8_GROUP) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "unknown form of output");
  if (!(p->eps >= 0.0f)) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "eps below zero");
  if (!p->residual != !p->sum) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "the residual and the place of the sum go together");
  const bool small = p->out != RINGAR_OUT_SAME;
  const size_t es = size_of(p->dtype), ws = size_of(p->param_dtype), ys = small ? 1 : es;
  const int64_t scales = !small ? 0 : p->out == RINGAR_OUT_FP8_ROW ? 1 : (p->cols + kScaleGroup - 1) / kScaleGroup;
  if (small && !p->scale && p->rows) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "scale is null");
  const int64_t added = p->residual ? p->rows : 0;
  TRY(check_mats({{"x", p->x, p->rows, p->cols, p->ldx, es, false, false, true},
                  {"residual", p->residual, added, p->cols, p->ldr, es, false, false, true},
                  VEC("weight", p->weight, p->cols, ws, false),
                  {"sum", p->sum, added, p->cols, p->lds, es, true},
                  {"y", p->y, p->rows, p->cols, p->ldy, ys, true},
                  {"scale", p->scale, scales ? p->rows : 0, scales, scales, 4, true},
                  VEC("rstd", p->rstd, p->rows, 4, true)}));
  if (p->rows == 0) return RINGAR_SUCCESS;
  RmsArgs a = {};
  a.x = p->x;
  a.residual = p->residual;
  a.weight = p->weight;
  a.sum = p->sum;
  a.y = p->y;
  a.scale = p->scale;
  a.rstd = p->rstd;
  a.ldx = p->ldx;
  a.ldr = p->ldr;
  a.lds = p->lds;
  a.ldy = p->ldy;
  a.rows = p->rows;
  a.cols = (int)p->cols;
  // a row of one group is a row of one scale
  a.out = scales == 1 ? kOutRow8 : p->out;
  a.scales = (int)scales;
  a.eps = p->eps;
  a.inv_cols = 1.0f / (float)p->cols;
  HIP_TRY(launch_rms_forward(p->dtype, p->param_dtype, a, (hipStream_t)stream));
  return RINGAR_SUCCESS;
}

static ringar_result_t rms_backward(const ringar_rms_norm_backward_t* p, ringar_stream_t stream) {
  if (!p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "null arguments");
  TRY(check_rms(p->dtype, p->param_dtype, p->rows, p->cols));
  const size_t es = size_of(p->dtype), ws = size_of(p->param_dtype);
  TRY(check_mats({{"dy", p->dy, p->rows, p->cols, p->lddy, es, false},
                  {"x", p->x, p->rows, p->cols, p->ldx, es, false},
                  {"rstd", p->rstd, 1, p->rows, p->rows, 4, false},
                  VEC("weight", p->weight, p->cols, ws, false),
                  {"dsum", p->dsum, p->dsum && p->dx ? p->rows : 0, p->cols, p->ldds, es, false, false, true},
                  {"dx", p->dx, p->dx ? p->rows : 0, p->cols, p->lddx, es, true},
                  VEC("dweight", p->dweight, p->cols, ws, true)}));
  if (!p->dweight && (!p->dx || p->rows == 0)) return RINGAR_SUCCESS;
  hipStream_t st = (hipStream_t)stream;
  RmsArgs a = {};
  a.x = p->x;
  a.dy = p->dy;
  a.weight = p->weight;
  a.residual = p->dx ? p->dsum : nullptr;
  a.y = p->dx;
  a.rstd = (float*)p->rstd;
  a.ldx = p->ldx;
  a.lddy = p->lddy;
  a.ldr = p->ldds;
  a.ldy = p->lddx;
  a.rows = p->rows;
  a.cols = (int)p->cols;
  a.inv_cols = 1.0f / (float)p->cols;
  a.blocks = rms_backward_blocks(p->rows, a.cols);
  std::lock_guard<std::mutex> lock(g_ws_mu);
  const bool split = p->dweight && (a.blocks != 1 || p->cols > kNormLongest);
  if (split) {
    char* ws_p = nullptr;
    TRY(workspace(st, (size_t)a.blocks * p->cols * 4, &ws_p));
    a.part = (float*)ws_p;
  } else {
    a.dweight = p->dweight;
  }
  if (p->rows) HIP_TRY(launch_rms_backward(p->dtype, p->param_dtype, a, st));
  if (split) HIP_TRY(launch_col_sum(p->param_dtype, {a.part, a.blocks, p->cols, p->cols, p->dweight, nullptr}, st));
  return RINGAR_SUCCESS;
}

static ringar_result_t drop(const ringar_dropout_t* p, ringar_stream_t stream) {
  if (!p) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "null arguments");
  if (!type_ok(p->dtype)) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "dropout takes fp16, bf16 or fp32");
  if (!dims_ok({p->rows, p->cols})) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "rows or cols out of range");
  if (!(p->p >= 0.0 && p->p <= 1.0)) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "p is a probability, 0 to 1");
  constexpr int64_t kWords = 1ll << 32;
  if (p->first_row < 0 || p->first_row > kWords - p->rows) return refuse(RINGAR_ERR_INVALID_ARGUMENT, "rows are counted in 32 bits");
  if (p->first_col < 0 || p->first_col % 8 || p->first_col > kMaxDim - p->cols)
    return refuse(RINGAR_ERR_INVALID_ARGUMENT, "first_col must be a multiple of 8 and the last column within 2^31 - 1025");
  const size_t es = size_of(p->dtype);
  const int64_t added = p->residual ? p->rows : 0;
  TRY(check_mats({{"x", p->x, p->rows, p->cols, p->ldx, es, false, true},
                  {"residual", p->residual, added, p->cols, p->ldr, es, false, true},
                  VEC("more_offset", p->more_offset, 1, 8, false),
                  {"y", p->y, p->rows, p->cols, p->ldy, es, true}}));
  if (p->rows == 0 || p->cols == 0) return RINGAR_SUCCESS;
  DropArgs a = {};
  a.x = p->x;
  a.residual = p->residual;
  a.y = p->y;
  a.more = p->more_offset;
  a.ldx = p->ldx;
  a.ldr = p->ldr;
  a.ldy = p->ldy;
  a.rows = p->rows;
  a.cols = (int)p->cols;
  a.first_row = p->first_row;
  a.first_block = (int)(p->first_col / 8);
  a.seed[0] = (uint32_t)p->seed;
  a.seed[1] = (uint32_t)(p->seed >> 32);
  a.offset = p->offset;
  a.threshold = (uint32_t)std::floor(p->p * 65536.0 + 0.5);
  a.scale = a.threshold < 65536 ? (float)(65536.0 / (65536.0 - a.threshold)) : 0.0f;
  HIP_TRY(launch_dropout(p->dtype, a, (hipStream_t)stream));
  return RINGAR_SUCCESS;
}

extern "C" {

ringar_result_t ringar_rms_norm(const ringar_rms_norm_t* args, ringar_stream_t stream) {
  return guarded([&] { return rms_forward(args, stream); });
}

ringar_result_t ringar_rms_norm_backward(const ringar_rms_norm_backward_t* args, ringar_stream_t stream) {
  return guarded([&] { return rms_backward(args, stream); });
}

ringar_result_t ringar_dropout(const ringar_dropout_t* args, ringar_stream_t stream) {
  return guarded([&] { return drop(args, stream); });
}

}  // extern "C"
