// Cross attention: how a call is cut into blocks, and the join of gradients
// whose sums were split.
#include <initializer_list>

#include "attn_types.h"

namespace ringar {

// Parts of what the backward kernels' blocks go along, `turns` of 32 rows of
// `turn` us each: one round of blocks on the 256 CUs after the other, and for
// parts a second launch and what it reads and writes (`part` bytes each).
static int splits_for(const AttnArgs& a, int64_t blocks, int64_t turns, double turn, double part) {
  double best = 0;
  int splits = 1;
  for (int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
    if (s > 1 && s > turns) break;
    const double rounds = (double)((blocks * s + 255) / 256);
    const double us = rounds * (double)((turns + s - 1) / s + 1) * turn + (s > 1 ? 4 + 0.3 * s + s * part * 2 / 4e6 : 0);
    if (best == 0 || us < 0.97 * best) {
      best = us;
      splits = s;
    }
  }
  return splits;
}

// Blocks of the grid: whole rounds of pieces over the XCDs.
int64_t attn_blocks(const AttnArgs& a) {
  const int64_t pieces = (int64_t)a.pieces * a.kv_heads * a.batch;
  return (pieces + 7) / 8 * 8 * a.piece;
}

// Pieces: a key head's blocks, or less where there are few key heads (64 pieces
// in all, then), of like sizes, as neighbours lie on different XCDs; single
// blocks where whole rounds would pass what a launch takes.
static void deal(AttnArgs& a) {
  const int64_t each = (int64_t)a.tiles * a.splits, groups = (int64_t)a.kv_heads * a.batch;
  const int64_t pieces = groups ? (64 + groups - 1) / groups : 1;
  a.pieces = (int)(pieces < each ? pieces : each);
  a.piece = a.pieces ? (int)((each + a.pieces - 1) / a.pieces) : 0;
  if (attn_blocks(a) > most_blocks(256)) {
    a.pieces = (int)each;
    a.piece = 1;
  }
}

// Columns that a kernel computes for head_dim.
static int padded(int dtype, int dim) { return dim <= 64 ? 64 : dtype == kF32 && dim <= 96 ? 96 : 128; }

// The forward pass's form and its parts along the keys: the one whose time, put
// together from what was measured over 1 .. 1024 queries, 500 .. 65536 keys, 1
// .. 64 sequences and 1 .. 20 heads, is the least.  In us:
//   a turn of one wave (32 rows, 32 keys): 0.33 at head_dim 64, 0.46 at 128, fp32
//   0.034 for each of 64, 96 or 128 columns (one wave a SIMD and two cost the same a turn: the clock drops);
//   of few rows, each wave's tiles on its own: 0.45 at least where other blocks
//   read them too, 0.75 where they come from memory;
//   start and end 5, of few rows' tiles side by side again for each further round of
//   blocks, 6 (one block a CU) and 3 at head_dim 64 (two; single tiles wait for
//   memory, which more blocks hide): 56 x 186 x 330, 4 heads of 64, bf16,
//   took 19 us in that form, which was chosen without this term, and 12 as
//   planned now; a second launch 3.5 and 0.3 a part, and the parts' bytes;
//   keys and values from memory once at 5 TB/s, and to every block at 18.
// Lengths, which are not known here, count as all keys.  (As three fourths of the
// bytes, in 40 shapes that this changes: with all keys 0.7% and with three fourths of
// them 2.8% less time, with a fourth 10% more; .66 .. 1.45 times the time of single ones.)
void plan_attn_forward(int dtype, AttnArgs& a) {
  const bool wide = dtype == kF32, far = a.dim > 64;
  const double bytes = 2.0 * a.keys * a.kv_heads * a.batch * a.dim * (wide ? 4 : 2);
  const double turn = wide ? 0.034 * padded(dtype, a.dim) : far ? 0.46 : 0.33;
  double best = 0;
  for (int form = a.rows <= 32 ? kFewRows : kManyRows; form <= kFewRows; form++) {
    if (form == kSomeRows && wide && far) continue;
    const int rows = form == kFewRows ? 32 : 128;
    const int groups = form == kManyRows ? 1 : form == kSomeRows ? 2 : wide && far ? 2 : 4;       // along the keys
    const int64_t tiles = ((int64_t)a.rows + rows - 1) / rows, units = tiles * a.kv_heads * a.batch;
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      if (splits > 1 && (int64_t)splits * 128 > a.keys) break;
      const double turns = (double)(((int64_t)a.keys + 32 * groups * splits - 1) / (32 * groups * splits));
      const double rounds = (double)((units * splits + 255) / 256);      // blocks of a CU
      double work = rounds * turns;
      if (form == kSomeRows) work *= rounds > 1 ? 2.0 : 1.8;
      const double wait = (form != kFewRows ? 0.0 : tiles > 1 ? 0.45 : 0.75) / rounds;
      work *= wait > turn ? wait : turn;
      if (form == kFewRows && tiles > 1) work += (rounds - 1) * (far ? 6 : 3);
      const double memory = bytes / 5e6 > bytes * tiles / 18e6 ? bytes / 5e6 : bytes * tiles / 18e6;
      double us = 5 + (work > memory ? work : memory);
      if (splits > 1) us += 3.5 + 0.3 * splits + (double)splits * a.rows * a.kv_heads * a.batch * a.dim * 8 / 4e6;
      if (best == 0 || us < 0.97 * best) {
        best = us;
        a.form = form;
        a.tiles = (int)tiles;
        a.splits = splits;
      }
    }
  }
  deal(a);
}

// (A turn's time as measured: 4 waves of 32 rows.)
void plan_attn_dq(int dtype, AttnArgs& a) {
  const bool far = a.dim > 64;
  a.tiles = (int)(((int64_t)a.rows + 127) / 128);
  a.splits = splits_for(a, (int64_t)a.tiles * a.kv_heads * a.batch, ((int64_t)a.keys + 31) / 32, dtype == kF32 ? 0.047 * padded(dtype, a.dim) : far ? 0.7 : 0.45,
                        4.0 * a.batch * a.heads * a.queries * a.dim);
  deal(a);
}

void plan_attn_dkv(int dtype, AttnArgs& a) {
  const bool far = a.dim > 64;
  a.tiles = (int)(((int64_t)a.keys + 127) / 128);
  a.splits = splits_for(a, (int64_t)a.tiles * a.kv_heads * a.batch, (int64_t)a.group * ((a.queries + 31) / 32), dtype == kF32 ? 0.062 * padded(dtype, a.dim) : far ? 1.0 : 0.6,
                        8.0 * a.batch * a.kv_heads * a.keys * a.dim);
  deal(a);
}

template <typename T> __global__ __launch_bounds__(256) void attn_join(AttnJoinArgs a) {
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < a.count * a.outs; at += (int64_t)gridDim.x * 1024) {
    const int which = at >= a.count;
    T* out = (T*)a.out[which] + (at - which * a.count);
    if (!a.out[which]) continue;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.splits; s++) {
      const Pack<float, 4> p = load_pack<float, 4>(a.part + s * (a.count * a.outs) + at);
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] += p.v[j];
    }
    Pack<T, 4> o;
#pragma unroll
    for (int j = 0; j < 4; j++) o.v[j] = (T)(v[j] * a.scale[which]);
    store_pack<T, 4>(out, o);
  }
}

hipError_t launch_attn_join(int dtype, const AttnJoinArgs& a, hipStream_t st) {
  const int64_t blocks = (a.count * a.outs / 4 + 255) / 256;
  const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
  if (dtype == kF32) return launch_kernel(attn_join<float>, grid, 256, st, a);
  if (dtype == kF16) return launch_kernel(attn_join<_Float16>, grid, 256, st, a);
  return launch_kernel(attn_join<__bf16>, grid, 256, st, a);
}

#define RINGAR_BY_TYPE(call)                       \
  do {                                             \
    if (dtype == kF32) return call<float>(a, st);  \
    if (dtype == kF16) return call<_Float16>(a, st); \
    return call<__bf16>(a, st);                    \
  } while (0)

hipError_t launch_attn_forward(int dtype, const AttnArgs& a, hipStream_t st) { RINGAR_BY_TYPE(attn_forward_of); }
hipError_t launch_attn_delta(int dtype, const AttnArgs& a, hipStream_t st) { RINGAR_BY_TYPE(attn_delta_of); }
hipError_t launch_attn_dq(int dtype, const AttnArgs& a, hipStream_t st) { RINGAR_BY_TYPE(attn_dq_of); }
hipError_t launch_attn_dkv(int dtype, const AttnArgs& a, hipStream_t st) { RINGAR_BY_TYPE(attn_dkv_of); }

}  // namespace ringar
