// Products by element type, and the rules that choose their kernel.
#include "block_types.h"

namespace ringar {

hipError_t launch_gemm_f16(int epi, const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_bf16(int epi, const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_f32(int epi, const GemmArgs& a, hipStream_t st);

namespace {

struct Tile {
  int m, n;
};
constexpr Tile kTiles[] = {{256, 256}, {128, 128}, {64, 128}, {128, 128}, {16, 16}};

// Operands the direct loads take: rows (or k lines) that start at 16-byte
// boundaries, and offsets within a tile that fit the loads' 32 bits.
bool operand_ok(const void* p, int64_t pitch, bool rows, int es, int64_t extra_rows) {
  const int64_t bytes = pitch * es;
  if ((uintptr_t)p % 16 || bytes % 16) return false;
  return ((rows ? 256 : 64) + extra_rows) * bytes < (1ll << 32) - 4096;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t tiles_of(int variant, int epi, const GemmArgs& a) {
  const Tile t = kTiles[variant];
  if (variant == kRows) return rows_tiles(epi, a.n);
  const int64_t cols = epi == kEpiGated ? 2 * (int64_t)a.n : a.n;
  return ceil_div(a.m, t.m) * ceil_div(cols, t.n);
}

}  // namespace

size_t plan_gemm(int dtype, int epi, GemmArgs& a) {
  a.splits = 1;
  a.k_per_split = a.k;
  a.variant = kStaged128;
  if (a.m == 0 || a.n == 0) return 0;
  const int es = dtype == kF32 ? 4 : 2;
  const bool arow = a.sak == 1, brow = a.sbk == 1;
  const int64_t wide = epi == kEpiGated ? 2 * (int64_t)a.n : a.n;
  const bool direct = operand_ok(a.a, arow ? a.sam : a.sak, arow, es, 0) &&
                     operand_ok(a.b, brow ? a.sbn : a.sbk, brow, es, epi == kEpiGated ? a.n : 0);
  const int step = 128 / es;
  a.variant = !direct ? kStaged128 : tiles_of(kTile256, epi, a) >= 192 && es == 2 ? kTile256 : arow && a.m <= 64 ? kTile64 : kTile128;
  if (epi != kEpiStore && a.m <= 16) {
    a.variant = kRows;
    // k over several blocks until there are two for every CU, each with
    // two steps for each of its 8 waves or more
    const int64_t tiles = rows_tiles(epi, a.n), turns = ceil_div(a.k, 8 * 256 / es);
    int64_t splits = tiles >= 256 ? 1 : ceil_div(512, tiles);
    if (splits > turns / 2) splits = turns / 2;
    if (splits < 1 || tiles > kCounters) splits = 1;
    const int64_t per = ceil_div(turns, splits) * (8 * 256 / es);
    a.k_per_split = (int)(per < a.k ? per : a.k);
    a.splits = a.k ? (int)ceil_div(a.k, per) : 1;
    return a.splits > 1 ? (size_t)tiles * a.splits * a.m * 16 * 4 : 0;
  }
  // parts of k: enough blocks to fill the GPU where the output has few tiles
  const int64_t tiles = tiles_of(a.variant, epi, a), steps = ceil_div(a.k, step);
  const int64_t want = a.variant == kTile256 ? 256 : 512;
  int64_t splits = tiles >= want / 2 || steps < 8 ? 1 : ceil_div(want, tiles);
  if (splits > steps / 4) splits = steps / 4;
  if (splits < 1) splits = 1;
  const int64_t per = ceil_div(steps, splits);
  a.k_per_split = (int)(per * step < a.k ? per * step : a.k);
  a.splits = (int)(steps ? ceil_div(steps, per) : 1);
  return a.splits > 1 ? (size_t)a.splits * a.m * wide * 4 : 0;
}

int64_t gemm_blocks(int dtype, int epi, const GemmArgs& a) {
  (void)dtype;
  return tiles_of(a.variant, epi, a) * a.splits;
}

hipError_t launch_gemm(int dtype, int epi, const GemmArgs& a, hipStream_t st) {
  if (dtype == kF16) return launch_gemm_f16(epi, a, st);
  if (dtype == kBF16) return launch_gemm_bf16(epi, a, st);
  return launch_gemm_f32(epi, a, st);
}

}  // namespace ringar
