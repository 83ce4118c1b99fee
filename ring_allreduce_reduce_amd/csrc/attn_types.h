// Kernel arguments of cross attention.
#pragma once

#include "block_types.h"

namespace ringar {

// rows of head_dim values: strides of the sequence, the row and the head, in elements
struct HeadRows {
  const void* p;
  int64_t batch, row, head;
};

// the forward kernel's blocks: 128 rows, 128 rows with two groups of waves along
// the keys, and 32 rows with all waves along the keys
enum : int { kManyRows = 0, kSomeRows = 1, kFewRows = 2 };

struct AttnArgs {
  HeadRows q, k, v;
  HeadRows y, dy;          // y: forward's output, backward's input
  const int32_t* lengths;  // or null
  float* lse;              // forward: or null; backward: an input
  int batch, queries, keys, heads, kv_heads, dim;
  int group;               // query heads of a key head
  int rows;                // group * queries: query rows that meet the same keys
  float scale;
  float scale2;            // scale log2(e)
  // set by the plan
  int tiles;               // blocks along the rows (dk, dv: the keys)
  int splits;              // parts of what a block goes along
  int piece, pieces;       // blocks of a piece, pieces of a key head's blocks
  int form;                // forward: how a block's waves share rows and keys
  float* part;             // splits > 1: [split][..] sums
  float* part_top;         // forward: [split][batch][kv head][row]: maximum, sum of exponentials
  float* lse2;             // backward: log2 of the rows' sums, and delta, batch x heads x queries
  float* delta;
  void *dq, *dk, *dv;      // contiguous
};

// one gradient, or two side by side, as sums of `splits` parts, in order
struct AttnJoinArgs {
  const float* part;       // [split][out][count]
  void* out[2];            // null: not wanted
  float scale[2];
  int64_t count;
  int outs;
  int splits;
};

int64_t attn_blocks(const AttnArgs& a);
void plan_attn_forward(int dtype, AttnArgs& a);
void plan_attn_dq(int dtype, AttnArgs& a);
void plan_attn_dkv(int dtype, AttnArgs& a);
hipError_t launch_attn_forward(int dtype, const AttnArgs& a, hipStream_t st);
hipError_t launch_attn_delta(int dtype, const AttnArgs& a, hipStream_t st);
hipError_t launch_attn_dq(int dtype, const AttnArgs& a, hipStream_t st);
hipError_t launch_attn_dkv(int dtype, const AttnArgs& a, hipStream_t st);
hipError_t launch_attn_join(int dtype, const AttnJoinArgs& a, hipStream_t st);

// one translation unit per type and pass
template <typename T> hipError_t attn_forward_of(const AttnArgs& a, hipStream_t st);
template <typename T> hipError_t attn_delta_of(const AttnArgs& a, hipStream_t st);
template <typename T> hipError_t attn_dq_of(const AttnArgs& a, hipStream_t st);
template <typename T> hipError_t attn_dkv_of(const AttnArgs& a, hipStream_t st);

}  // namespace ringar
