// Products by element type, and the rules that choose their kernel.
#include "block_types.h"
#include "op_checks.h"

namespace ringar {

hipError_t launch_gemm_f16(int epi, const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_bf16(int epi, const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_f32(int epi, const GemmArgs& a, hipStream_t st);
hipError_t launch_gradients_f16(const GemmArgs& x, const GemmArgs& w, const ColSumArgs& sums, hipStream_t st);
hipError_t launch_gradients_bf16(const GemmArgs& x, const GemmArgs& w, const ColSumArgs& sums, hipStream_t st);
hipError_t launch_gradients_f32(const GemmArgs& x, const GemmArgs& w, const ColSumArgs& sums, hipStream_t st);

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Operands the direct loads take: rows (or k lines) that start at 16-byte
// boundaries, and offsets within a tile that fit the loads' 32 bits.
bool operand_ok(const void* p, int64_t pitch, bool rows, int es, int64_t extra_rows) {
  const int64_t bytes = pitch * es;
  if ((uintptr_t)p % 16 || bytes % 16) return false;
  return ((rows ? 256 : 64) + extra_rows) * bytes < (1ll << 32) - 4096;
}

struct Tile {
  int m, n;
};
Tile tile_of(int variant, int epi) {
  switch (variant) {
    case kTile256: return {256, 256};
    case kTile128: return {128, 128};
    default: return {64, epi == kEpiGated ? 128 : 64};
  }
}

int64_t tiles_of(int variant, int epi, const GemmArgs& a) {
  if (variant == kRows) return rows_tiles(epi, a.n);
  const Tile t = tile_of(variant, epi);
  return ceil_div(a.m, t.m) * ceil_div(epi == kEpiGated ? 2 * (int64_t)a.n : a.n, t.n);
}

// Microseconds of a tiled launch: a start, and for every step of 128 bytes of
// k (and one and a half more, to fill the buffers and to finish) either a lone
// block's latency or the CU's throughput, whichever is more.
// Measured on MI355X over 32 .. 2500 rows, widths of 1024 .. 4096 and splits
// of 1 .. 16 (bf16 and fp32, the fastest choice of this table within 10% of
// the fastest measured): a 64 x 64 tile wins until its blocks are about four
// to a CU (512 x 4096 x 4096 bf16: 26 us, 128 x 128 34 us), 256 x 256 from
// about 200 tiles on (8192 x 8192 x 8192: 0.87 ms).
struct Cost {
  double start, alone, shared;
};
Cost cost_of(int variant, int epi, int es, bool arow, bool brow) {
  if (es == 4) {
    if (variant == kTile128) return {1, 1.95, 1.95};
    if (variant == kTile64) return epi == kEpiGated ? Cost{2, 1.06, 1.0} : Cost{2, 0.6, 0.51};
    return epi == kEpiGated ? Cost{2, 1.4, 1.3} : Cost{2, 0.8, 0.7};
  }
  switch (variant) {
    case kTile256: return {6, 1.43, 1.43};
    case kTile128: return {2.6, 0.6, 0.55};
    case kTile64: return epi == kEpiGated ? Cost{2.6, 0.31, 0.29} : arow ? Cost{2.6, 0.24, 0.18} : Cost{2.6, 0.25, 0.23};
    default: return epi == kEpiGated ? Cost{2, 1.0, 0.6} : brow ? Cost{2, 0.95, 0.45} : Cost{2, 0.95, 0.6};
  }
}

struct Choice {
  int variant, splits;
  double us;
};

// 256 x 256 tiles run one to a CU: a few left over for a last round are done
// in quarters by 128 x 128 blocks, which take less than half as long (2500 x
// 4096 x 2 * 10240 bf16: 800 tiles, 32 of them in quarters).  Both run in one
// launch, whose blocks must be few enough for it.
int tail_of(int variant, int splits, int64_t tiles) {
  const int left = (int)(tiles % 256);
  return variant == kTile256 && splits == 1 && tiles > 256 && tiles < most_blocks(512) - 256 && left <= 64 ? left : 0;
}

// The cheapest split of one kernel: parts of k fill the GPU where the output
// has few tiles, and cost a pass over the parts.
Choice cheapest(int variant, int epi, int es, const GemmArgs& a) {
  const Cost c = cost_of(variant, epi, es, a.sak == 1, a.sbk == 1);
  const int64_t tiles = tiles_of(variant, epi, a), steps = ceil_div(a.k, 128 / es);
  const double outputs = (double)a.m * a.n * (epi == kEpiGated ? 2 : 1);
  // what comes from memory at 5 TB/s at best
  const double memory = ((double)a.m * a.k + (double)a.k * a.n * (epi == kEpiGated ? 2 : 1) + (double)a.m * a.n) * es / 5e6;
  Choice best = {variant, 1, 0};
  for (int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
    if (s > 1 && steps < 2 * s) break;
    const int64_t per = ceil_div(steps, s);
    const double at_once = c.shared * (double)ceil_div(tiles * s, 256);
    double us = (per + 1.5) * (at_once > c.alone ? at_once : c.alone);
    us = c.start + (us > memory ? us : memory) + (s > 1 ? 4.5 + outputs * s * 8 / 8e6 : 0);
    if (tail_of(variant, s, tiles)) us += (per + 1.5) * (cost_of(kTile128, epi, es, true, true).alone - c.shared);
    if (s == 1 || us < best.us) best = {variant, s, us};
  }
  return best;
}

// Rows up to which the forward product streams the weight (kRows), `direct`:
// the tiles could load both operands as they lie.  Measured over 1 .. 16 rows, k of
// 64 .. 8192 and 1024 .. 65536 weight rows (gated: both), us of the tiles and of the
// stream:
//   fp32: the stream wins everywhere but at k = 64 with 32768 rows or more (6.0,
//     7.3): 16 x 4096 x 4096 24.3, 19.3; x 16384 74.5, 64.4; 8 x 4095 x 16384 81, 62.
//   16 bits, few weight rows: the stream (16 x 2048 x 4096: 10.6, 6.2; 16 x 1024 x
//     8192: 7.2, 6.3).
//   many of them, 9 rows and more: the tiles, which read the rows once for 128
//     columns (16 x 4096 x 20480: 37.6, 42.6; at 9 rows equal, 37.2, 36.0).
//   many of them, a short k: the stream's blocks end as soon as they have
//     started (4 x 1024 x 16384: 7.7, 8.7; 8 x 256 x 65536: 8.8, 14.3; 8 x 2048 x
//     65536: 59.7, 54.4); not where the tiles would need a copy (4 x 1023 x 16384: 16.2, 11.5).
int most_rows(int es, int64_t k, int64_t wide, bool direct) {
  if (es == 4 || wide < 12288) return 16;
  if (k <= 1024 && direct) return 0;
  return wide < 16384 ? 16 : 8;
}

}  // namespace

// `only`: the one tiled kernel to consider, or -1.
static GemmPlan plan_tiles(int dtype, int epi, const GemmArgs& given, int only, Choice* chosen) {
  GemmPlan p = {};
  p.epi = epi;
  p.args = given;
  GemmArgs& a = p.args;
  a.splits = 1;
  a.k_per_split = a.k;
  a.variant = kStaged64;
  if (a.m == 0 || a.n == 0) return p;
  const int es = dtype == kF32 ? 4 : 2;
  const int64_t wide = epi == kEpiGated ? 2 * (int64_t)a.n : a.n;
  const bool arow = a.sak == 1, brow = a.sbk == 1;
  const bool ok_a = operand_ok(a.a, arow ? a.sam : a.sak, arow, es, 0);
  const bool ok_b = operand_ok(a.b, brow ? a.sbn : a.sbk, brow, es, epi == kEpiGated ? a.n : 0);
  if (epi != kEpiStore && a.k >= 16 / es && a.m <= most_rows(es, a.k, wide, ok_a && ok_b)) {
    a.variant = kRows;
    // k over several blocks until there are two for every CU, each with
    // two steps for each of its 8 waves or more
    const int64_t turn = 8 * 256 / es, tiles = rows_tiles(epi, a.n), turns = ceil_div(a.k, turn);
    int64_t splits = tiles >= 256 ? 1 : ceil_div(512, tiles);
    if (splits > turns / 2) splits = turns / 2;
    if (splits < 1 || tiles > kCounters) splits = 1;
    const int64_t per = ceil_div(turns, splits) * turn;
    a.k_per_split = (int)(per < a.k ? per : a.k);
    a.splits = a.k ? (int)ceil_div(a.k, per) : 1;
    a.tile_count = (int)tiles;
    p.bytes = a.splits > 1 ? (size_t)tiles * a.splits * a.m * 16 * 4 : 0;
    return p;
  }
  // the operands as stored, and copies with padded rows
  const int64_t rows_a = arow ? a.m : a.k, cols_a = arow ? a.k : a.m, rows_b = brow ? wide : a.k, cols_b = brow ? a.k : wide;
  const int64_t pad = 128 / es;
  p.packed_a = ceil_div(cols_a, pad) * pad;
  p.packed_b = ceil_div(cols_b, pad) * pad;
  auto copy_us = [&](int64_t rows, int64_t pitch) { return (double)rows * pitch * es * 2 / 4.5e6; };
  Choice best = cheapest(only < 0 ? kTile64 : only, epi, es, a);
  for (int v : {kTile128, kTile256}) {
    if (only >= 0 || (v == kTile256 && es == 4)) continue;
    const Choice c = cheapest(v, epi, es, a);
    if (c.us < best.us) best = c;
  }
  if (!ok_a || !ok_b) {
    const double copies = 3.5 + (ok_a ? 0 : copy_us(rows_a, p.packed_a)) + (ok_b ? 0 : copy_us(rows_b, p.packed_b));
    const int64_t packs = (ok_a ? 0 : rows_a * p.packed_a) + (ok_b ? 0 : rows_b * p.packed_b);
    const bool fits = packs / (16 / es) / 256 < most_blocks(256) - 2 && ((arow ? 256 : 64) * p.packed_a + 64) * es < (1ll << 32) - 4096 &&
                      ((brow ? 256 + (epi == kEpiGated ? a.n : 0) : 64) * p.packed_b + 64) * es < (1ll << 32) - 4096;
    const Choice staged = cheapest(kStaged64, epi, es, a);
    best.us += copies;
    if (fits && best.us < staged.us) {
      p.pack_a = !ok_a;
      p.pack_b = !ok_b;
    } else {
      best = staged;
    }
  }
  *chosen = best;
  a.variant = best.variant;
  const int64_t step = 128 / es, steps = ceil_div(a.k, step), per = ceil_div(steps, best.splits);
  a.k_per_split = (int)(per * step < a.k ? per * step : a.k);
  a.splits = (int)(steps ? ceil_div(steps, per) : 1);
  const int64_t tiles = tiles_of(a.variant, epi, a);
  if (tiles * a.splits > 0x7fffffff - 1024) {
    p.too_many = true;
    return p;
  }
  a.tail_count = tail_of(a.variant, a.splits, tiles);
  a.tile_count = (int)tiles - a.tail_count;
  auto part = [&](size_t n) { p.bytes += (n + 255) / 256 * 256; };
  if (a.splits > 1) part((size_t)a.splits * a.m * wide * 4);
  if (p.pack_a) part((size_t)rows_a * p.packed_a * es);
  if (p.pack_b) part((size_t)rows_b * p.packed_b * es);
  return p;
}

GemmPlan plan_gemm(int dtype, int epi, const GemmArgs& a) {
  Choice c = {};
  return plan_tiles(dtype, epi, a, -1, &c);
}

bool plan_gradients(int dtype, const GemmArgs& x, const GemmArgs& w, GemmPlan* px, GemmPlan* pw) {
  Choice cx = {}, cw = {};
  *px = plan_tiles(dtype, kEpiStore, x, -1, &cx);
  *pw = plan_tiles(dtype, kEpiStore, w, -1, &cw);
  if (!x.m || !x.n || !w.m || !w.n || px->too_many || pw->too_many) return false;
  const int es = dtype == kF32 ? 4 : 2;
  double best = cx.us + cw.us;
  bool together = false;
  for (int v : {kTile64, kTile128}) {
    Choice tx = {}, tw = {};
    const GemmPlan qx = plan_tiles(dtype, kEpiStore, x, v, &tx), qw = plan_tiles(dtype, kEpiStore, w, v, &tw);
    if (qx.args.variant != v || qw.args.variant != v || qx.too_many || qw.too_many) continue;
    // one launch, with a block for every 64 of the bias's column sums
    const int64_t blocks = (int64_t)qx.args.tile_count * qx.args.splits + (int64_t)qw.args.tile_count * qw.args.splits + w.m / 64 + 1;
    if (blocks > most_blocks(v == kTile128 ? 512 : 256)) continue;
    // The blocks share the CUs: the longer product's time alone, or all their
    // steps at the CU's throughput; a start and a launch less.
    const Cost c = cost_of(v, kEpiStore, es, true, false);
    auto steps = [&](const GemmArgs& a) { return (double)a.tile_count * a.splits * (a.k_per_split / (128.0 / es) + 1.5); };
    const double shared = c.start + (steps(qx.args) + steps(qw.args)) * c.shared / 256;
    const double alone = tx.us > tw.us ? tx.us : tw.us;
    const double joins = (qx.args.splits > 1 ? 4.5 : 0) + (qw.args.splits > 1 ? 4.5 : 0) + (qx.pack_a || qx.pack_b ? 3.5 : 0) +
                         (qw.pack_a || qw.pack_b ? 3.5 : 0);
    const double us = (shared > alone ? shared : alone) + (shared > alone ? joins : 0);
    if (us >= best) continue;
    best = us;
    *px = qx;
    *pw = qw;
    together = true;
  }
  return together;
}

// The planned product's arguments with its workspace in place and its copies
// enqueued.
static hipError_t prepare(int dtype, const GemmPlan& p, char* ws, uint32_t* counters, hipStream_t st, GemmArgs* out) {
  GemmArgs a = p.args;
  const int es = dtype == kF32 ? 4 : 2;
  const int64_t wide = p.epi == kEpiGated ? 2 * (int64_t)a.n : a.n;
  auto part = [&](size_t n) {
    char* at = ws;
    ws += (n + 255) / 256 * 256;
    return at;
  };
  a.part = (float*)ws;
  a.arrived = counters;
  if (a.variant != kRows && a.splits > 1) a.part = (float*)part((size_t)a.splits * a.m * wide * 4);
  PackArgs packs = {};
  int count = 0;
  auto pack = [&](const void** from, int64_t* pitch, int64_t packed, int64_t rows, int64_t cols) {
    void* to = part((size_t)rows * packed * es);
    packs.one[count++] = {*from, to, *pitch, packed, rows, (int)cols, 0};
    *from = to;
    *pitch = packed;
  };
  if (p.pack_a) a.sak == 1 ? pack(&a.a, &a.sam, p.packed_a, a.m, a.k) : pack(&a.a, &a.sak, p.packed_a, a.k, a.m);
  if (p.pack_b) a.sbk == 1 ? pack(&a.b, &a.sbn, p.packed_b, wide, a.k) : pack(&a.b, &a.sbk, p.packed_b, a.k, wide);
  if (count == 1) {                  // no second copy: one without rows
    packs.one[1] = packs.one[0];
    packs.one[1].rows = 0;
  }
  const hipError_t e = count ? launch_pack(dtype, packs, st) : hipSuccess;
  *out = a;
  return e;
}

hipError_t launch_gemm(int dtype, const GemmPlan& p, char* ws, uint32_t* counters, hipStream_t st) {
  if (p.args.m == 0 || p.args.n == 0) return hipSuccess;
  GemmArgs a;
  const hipError_t e = prepare(dtype, p, ws, counters, st, &a);
  if (e != hipSuccess) return e;
  if (dtype == kF16) return launch_gemm_f16(p.epi, a, st);
  if (dtype == kBF16) return launch_gemm_bf16(p.epi, a, st);
  return launch_gemm_f32(p.epi, a, st);
}

hipError_t launch_gradients(int dtype, const GemmPlan& x, const GemmPlan& w, const ColSumArgs& sums, char* ws_x, char* ws_w, hipStream_t st) {
  GemmArgs ax, aw;
  hipError_t e = prepare(dtype, x, ws_x, nullptr, st, &ax);
  if (e == hipSuccess) e = prepare(dtype, w, ws_w, nullptr, st, &aw);
  if (e != hipSuccess) return e;
  if (dtype == kF16) return launch_gradients_f16(ax, aw, sums, st);
  if (dtype == kBF16) return launch_gradients_bf16(ax, aw, sums, st);
  return launch_gradients_f32(ax, aw, sums, st);
}

}  // namespace ringar
