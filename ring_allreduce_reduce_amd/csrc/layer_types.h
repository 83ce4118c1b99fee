// Kernel arguments of the root-mean-square norm and of dropout.
#pragma once

#include "block_types.h"

namespace ringar {

// Columns of a scale's group, and the 8-bit type's largest value (4 bits of
// exponent, 3 of mantissa, no infinity).
constexpr int kScaleGroup = 128;
constexpr float kLargest8 = 448.0f;
// A scale below this would have no finite reciprocal.
constexpr float kLeastScale = 0x1p-126f;

// what a norm's output is held in: x's type, or 8 bits with one scale a row,
// or one for every kScaleGroup columns
enum : int { kOutSame = 0, kOutRow8 = 1, kOutGroup8 = 2 };

struct RmsArgs {
  const void* x;
  const void* residual;  // or null.  Backward: the gradient of the sum, or null
  const void* dy;        // backward
  const void* weight;    // null: ones
  void* sum;             // with a residual: x + residual
  void* y;               // backward: dx (may be null)
  float* scale;          // 8 bits: [rows][groups]
  float* rstd;           // forward: may be null; backward: an input
  float* part;           // backward: [blocks][cols] sums, or null
  void* dweight;         // backward, without part: the sums of the one block, or null
  int64_t ldx, ldr, lddy, lds, ldy;
  int64_t rows;
  int cols;
  int blocks;            // of the backward grid
  int out;               // kOut..
  int scales;            // of a row
  float eps;
  float inv_cols;
  bool stream;           // outputs go past the caches
};

struct DropArgs {
  const void* x;
  const void* residual;  // or null
  void* y;
  const int64_t* more;   // added to the offset, or null
  int64_t ldx, ldr, ldy;
  int64_t rows;
  int64_t first_row;
  int cols;
  int first_block;       // first column / 8
  uint32_t seed[2];
  uint64_t offset;
  uint32_t threshold;    // values whose number is below are dropped
  float scale;
  // set by the launcher: a thread's step over the 8-column blocks of the rows
  int blocks;
  int step_blocks;
  int64_t step_rows;
};

hipError_t launch_rms_forward(int dtype, int wdtype, const RmsArgs& a, hipStream_t st);
int rms_backward_blocks(int64_t rows, int cols);
hipError_t launch_rms_backward(int dtype, int wdtype, const RmsArgs& a, hipStream_t st);
hipError_t launch_dropout(int dtype, const DropArgs& a, hipStream_t st);

}  // namespace ringar
