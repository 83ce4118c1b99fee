// Cross attention, backward.
//
//   P = exp(s - lse),  dP = dy v^T,  delta = sum dy y,  dS = P (dP - delta)
//   dq = scale dS k,  dk = scale dS^T q,  dv = P^T dy
//
// Two kernels, each of which computes S and dP again for what it sums over, so
// that every gradient is added up in one block's registers, in an order that
// is always the same (no atomics): 7 products in place of 5.
//   dq: a wave holds 32 query rows (Q, dy in fragments, dq^T in result
//   registers) and goes along the keys; S^T and dP^T have a row a lane.
//   dk, dv: a wave holds 32 keys (K, V in fragments, dk^T and dv^T in result
//   registers) and goes along the query rows of every head that shares them;
//   S and dP have a key a lane.
// P and dS are the next product's operand as they stand (attn_tile.h), rounded
// to the operands' type: what the matrix instructions take.  fp16 holds P times
// 2^10 where it meets dy, so that the small P of long rows keep their bits, and dS
// times a power of two that goes by its size.
//
// Times are medians, ranges two GPUs.  8 x 1024 x 2048, 16 heads of 128, bf16: dq 203
// .. 208 us, dk and dv 291 .. 301 (991 .. 1017 and 912 .. 945 TFLOP/s of what they
// compute).  Tried for dk, dv and not kept:
// 64 keys a wave with fragments read ahead by hand (408 us), 32 keys with them
// (321), values in fragments and longer query tiles (289, where the kept form took
// 281 in the same run; between runs it takes 281 .. 291).
#pragma once

#include "attn_tile.h"

namespace ringar {

template <typename T> struct Shift {
  static constexpr float kLog2 = sizeof(T) == 2 && !std::is_same_v<T, __bf16> ? 10.0f : 0.0f;
  static constexpr float kBack = kLog2 > 0.0f ? 0x1p-10f : 1.0f;
};

// lse in powers of two; +infinity where a row has no keys, so that its P are 0
__device__ inline float powers_of_two(float lse) { return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f; }

// dS = P (dP - delta) is as small as P and dy together: in fp16, whose steps below
// 2^-14 are 2^-24, it would lose most of its bits with dy near 1e-4 and some
// thousand keys.  So fp16 holds dS times a power of two, which is taken out of the
// fp32 sums again (both exact).  dq has one for each row, dk one for a wave's 32
// keys; each kernel says how it is found.  fp16 operands bound dP and delta by 2^39,
// so dS 2^60 is finite in fp32, and where all dS are 0 the power is that.
// (8 x 1024 x 2048, 16 heads, fp16, dq and dk with dv, without the powers and with
// them: head_dim 128 212 / 214 and 327 / 331 us, 64 124 / 125 and 182 / 186.)
template <typename T> constexpr bool kScaledSlopes = sizeof(T) == 2 && !std::is_same_v<T, __bf16>;
constexpr int kMostUp = 60;
__device__ inline float power_of_two(int n) { return __builtin_ldexpf(1.0f, n); }
// v = m 2^this, m in [1/2, 1); v is finite and not zero
__device__ inline int exponent_of(float v) { return __builtin_amdgcn_frexp_expf(v); }

// The lane's half of the sum of dy y over a row, in the order of its fragments.
template <typename Frag, int N> __device__ inline float half_delta(const Frag (&dy)[N], const Frag (&y)[N]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++)
#pragma unroll
    for (int j = 0; j < 16 / (int)sizeof(dy[0][0]); j++) s = fmaf((float)dy[i][j], (float)y[i][j], s);
  return s;
}

// lse2 and delta where no dq is wanted, whose kernel leaves them otherwise: the
// same sums, 32 rows a wave.
template <typename T> __global__ __launch_bounds__(256) void attn_delta(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t rows = (int64_t)a.batch * a.heads * a.queries;
  for (int64_t i = (int64_t)blockIdx.x * 128 + (threadIdx.x >> 6) * 32 + (lane & 31); i < rows; i += (int64_t)gridDim.x * 128) {
    const int64_t query = i % a.queries, bh = i / a.queries, head = bh % a.heads, batch = bh / a.heads;
    RowFrags<T, 128> dy, y;
    dy.load(row_at<T>(a.dy, batch, head, query), true, a.dim, lane);
    y.load(row_at<T>(a.y, batch, head, query), true, a.dim, lane);
    float s = half_delta(dy.f, y.f);
    s += __shfl_xor(s, 32);
    if (lane < 32) {
      a.lse2[i] = powers_of_two(a.lse[i]);
      a.delta[i] = s;
    }
  }
}

// ------------------------------------------------------------------------ dq
// As the forward pass, a wave works on three tiles (32 keys) at once: dS k of
// tile t - 1 and q k^T, dy v^T of tile t + 1 on the matrix units, dS of tile t on
// the vector units.  Four buffers in turn hold a tile from its loads, two turns
// ahead, to its last product.  delta comes from y's rows, a lane's half of one
// each, and is left for the other kernel with lse in powers of two.
//
// fp16's power of two: P is 1 at most, so a row's dS are bounded by the largest |dP
// - delta|, which the first tile's 32 keys stand for: below 2^10 there.  A later one
// 2^6 times as large may overflow, which leaves no column of the row finite: the
// block then takes its keys again, such rows at 2^-10 of their power, and once more at
// their natural size.  (Kept out of the loop, where a look for the largest dS and
// the sums' scaling spilled 116 registers at head_dim 128.)
template <typename T, int D> struct AttnDq {
  using M = Mma32<T>;
  using Frag = typename M::Frag;
  static constexpr int NW = 4, kThreads = 64 * NW, KT = 32;
  using Tile = RowTile<T, D, KT, NW>;
  static constexpr int kSteps = D / M::kK, kDims = D / 32;
  static constexpr int kShared = 8 * Tile::kPlace;
  static constexpr int kBlocksPerCu = D * sizeof(T) > 256 ? 1 : 2;     // registers

  static __device__ inline void run(const AttnArgs& a, char* smem) {
    const AttnPlace at(a);
    if (!at.valid) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = (at.tile * NW + wave) * 32 + (lane & 31);
    const bool exists = r < a.rows;
    const int r_in = exists ? r : a.rows - 1;
    const int head = at.head(a, r_in), query = r_in % a.queries;

    const int all = (at.length + KT - 1) / KT, per = (all + a.splits - 1) / a.splits;
    const int first = at.split * per, last = first + per < all ? first + per : all;
    const int turns = last - first, row_bytes = a.dim * (int)sizeof(T);
    const int64_t pitch_k = a.k.row * (int64_t)sizeof(T), pitch_v = a.v.row * (int64_t)sizeof(T);
    RowFrags<T, D> q, dy;
    q.load(row_at<T>(a.q, at.batch, head, query), exists, a.dim, lane);
    dy.load(row_at<T>(a.dy, at.batch, head, query), exists, a.dim, lane);
    float delta = 0.0f;
    {
      RowFrags<T, D> y;
      y.load(row_at<T>(a.y, at.batch, head, query), exists, a.dim, lane);
      delta = half_delta(dy.f, y.f);
      delta += __shfl_xor(delta, 32);
    }
    const int64_t stat = ((int64_t)at.batch * a.heads + head) * a.queries + query;
    const float lse2 = powers_of_two(a.lse[stat]);
    if (exists && lane < 32 && at.split == 0) {
      a.lse2[stat] = lse2;
      a.delta[stat] = delta;
    }

    RowStream keys, values;
    keys.start(row_at<T>(a.k, at.batch, at.kv_head, 0), pitch_k, (int64_t)first * KT, at.length, KT, row_bytes);
    values.start(row_at<T>(a.v, at.batch, at.kv_head, 0), pitch_v, (int64_t)first * KT, at.length, KT, row_bytes);
    Tile tk, tv;
    tk.start(pitch_k, a.dim, wave, lane);
    tv.start(pitch_v, a.dim, wave, lane);
    auto issue = [&](int turn) {              // of the turns in order
      if (turn >= turns) return;
      char* lds = smem + (turn & 3) * Tile::kPlace;
      tk.load(keys.next(), lds, wave);
      tv.load(values.next(), lds + 4 * Tile::kPlace, wave);
    };

    FragReader<T, KT> read(smem, lane);
    read.move_cols(2 * Tile::kPlace);         // rows of the buffer at hand, columns of that two turns back
    constexpr int kMmaQ = 32 / M::kK * kDims, kMma = kMmaQ + 2 * kSteps, kAhead = 3, kFrags = 32 / M::kK;
    f32x16 acc[kDims], s, dp, begun_s, begun_dp;
    Frag kf[kAhead], ds[kFrags], ds_next[kFrags];
#pragma unroll
    for (int i = 0; i < kDims; i++) acc[i] = zero16();
    // the turn's matrix instructions: dS k, then q k^T and dy v^T but for their last step
    auto frag = [&](int m) {
      if (m < kMmaQ) return read.cols(0, m / kDims * M::kK, m % kDims * 32);
      return read.rows((m - kMmaQ) & 1 ? 4 * Tile::kPlace : 0, 0, (m - kMmaQ) / 2);
    };
    auto products = [&](int from, int to, auto before, auto with) {
#pragma unroll
      for (int m = 0; m < kAhead; m++) kf[(from + m) % kAhead] = frag(from + m);
      before();
      if (to > kMmaQ) begun_s = begun_dp = zero16();
#pragma unroll
      for (int m = from; m < to; m++) {
        const int n = m - kMmaQ;
        if (m < kMmaQ) acc[m % kDims] = M::run(kf[m % kAhead], ds[m / kDims], acc[m % kDims]);
        else if (n & 1) begun_dp = M::run(kf[m % kAhead], dy.f[n / 2], begun_dp);
        else begun_s = M::run(kf[m % kAhead], q.f[n / 2], begun_s);
        if (m + kAhead < kMma && (to > kMmaQ || m + kAhead < kMmaQ)) kf[m % kAhead] = frag(m + kAhead);
        with(m);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto end_scores = [&] {
      s = M::run(kf[(kMma - 2) % kAhead], q.f[kSteps - 1], begun_s);
      dp = M::run(kf[(kMma - 1) % kAhead], dy.f[kSteps - 1], begun_dp);
    };
    constexpr int kEach = 16 / sizeof(T);
    float times = 1.0f, delta_up = delta;     // what dS is held times, and delta so
    auto slope = [&](Frag* to, int i) {
      const float away = kScaledSlopes<T> ? fmaf(dp[i], times, -delta_up) : dp[i] - delta;
      to[i / kEach][i % kEach] = (T)(fast_exp2(fmaf(s[i], a.scale2, -lse2)) * away);
      if (i % kEach == kEach - 1) asm volatile("" : "+v"(to[i / kEach]));
    };
    auto slopes = [&](int left) {             // of a tile with `left` keys
      // (computed here: sixteen rows or results kept from before the loop cost registers)
      int lane_now = lane;
      asm volatile("" : "+s"(left), "+v"(lane_now));
#pragma unroll
      for (int i = 0; i < 16; i++) {
        slope(ds, i);
        if (result_row(i, lane_now) >= left) ds[i / kEach][i % kEach] = (T)0.0f;
      }
    };
    auto hold_by_first = [&] {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; i++) most = fmaxf(most, fabsf(dp[i] - delta_up));
      most = fmaxf(most, __shfl_xor(most, 32));
      const int up = 10 - (most < INFINITY ? exponent_of(most) : 10);
      times = power_of_two(most > 0.0f && up < kMostUp ? up : kMostUp);
      delta_up *= times;
    };
    // whether any of the block's lanes says so; what lies in LDS is not needed any more
    auto any_of_block = [&](bool yes) {
      uint32_t* said = (uint32_t*)smem;
      const uint32_t of_wave = __any(yes);
      wait_lds();
      block_barrier();
      if (lane == 0) said[wave] = of_wave;
      wait_lds();
      block_barrier();
      uint32_t all = 0;
#pragma unroll
      for (int i = 0; i < NW; i++) all |= said[i];
      all = __builtin_amdgcn_readfirstlane(all);
      wait_lds();
      block_barrier();
      return all != 0;
    };
    auto nothing = [](int) {};
    auto start = [&](int turn) {
      wait_lds();
      block_barrier();
      issue(turn + 2);
      read.other((turn & 1 ? 3 : 1) * Tile::kPlace);      // on to buffer (turn + 1) % 4
    };
    // (the lane's row once more: kept over the loop it cost a register)
    auto row_now = [&] {
      int lane_now = lane;
      asm volatile("" : "+v"(lane_now));
      return (at.tile * NW + wave) * 32 + (lane_now & 31);
    };
    const int left = at.length - (last - 1) * KT, whole = left < KT ? turns - 1 : turns;
#pragma unroll 1
    for (int taken = 0; turns > 0; taken++) {
      issue(0);
      issue(1);
      if (turns > 1) wait_lds<2 * Tile::kLoads>();
      else wait_lds();
      block_barrier();
      products(kMmaQ, kMma - 2, [] {}, nothing);
      end_scores();
      if (kScaledSlopes<T> && taken == 0) hold_by_first();
      start(0);
      slopes(turns == 1 ? left : KT);
      if (turns > 1) {
        products(kMmaQ, kMma - 2, [] {}, nothing);
        end_scores();
      }
      for (int turn = 1; turn < whole; turn++) {
        start(turn);
        products(0, kMma - 2,                 // (after the last tile: scores of what lies there, not used)
                 [&] {
#pragma unroll
                   for (int i = 0; i < 2; i++) slope(ds_next, i);
                 },
                 [&](int m) {
#pragma unroll
                   for (int i = 2; i < 16; i++)
                     if ((i - 2) * (kMma - 2) / 14 == m) slope(ds_next, i);
                 });
#pragma unroll
        for (int f = 0; f < kFrags; f++) ds[f] = ds_next[f];
        end_scores();
      }
      if (turns > 1 && whole < turns) {
        start(whole);
        products(0, kMmaQ, [] {}, nothing);
        slopes(left);
      }
      read.other((turns & 1 ? 3 : 1) * Tile::kPlace);
      products(0, kMmaQ, [] {}, nothing);
      if (!kScaledSlopes<T> || taken == 2) break;
      // (a row whose delta is not finite cannot be helped)
      const bool over = row_now() < a.rows && fabsf(delta_up) < INFINITY && !(fabsf(acc[0][0]) < INFINITY);
      if (!any_of_block(over)) break;
      const float by = !over ? 1.0f : taken == 0 ? 0x1p-10f : times > 1.0f ? power_of_two(1 - exponent_of(times)) : 1.0f;
      times *= by;
      delta_up *= by;
      keys.back(turns);
      values.back(turns);
      read.other(((turns + 1) & 3) * Tile::kPlace);         // on to the first buffer
#pragma unroll
      for (int i = 0; i < kDims; i++) acc[i] = zero16();
    }
    const int r_out = row_now();
    if (r_out >= a.rows) return;
    if constexpr (kScaledSlopes<T>) {
      const float down = power_of_two(1 - exponent_of(times));
#pragma unroll
      for (int i = 0; i < kDims; i++) acc[i] *= down;
    }
    int queries = a.queries;                  // (a divisor of its own, for the same reason)
    asm volatile("" : "+s"(queries));
    const int64_t out = (((int64_t)at.batch * queries + r_out % queries) * a.heads + at.kv_head * a.group + r_out / queries) * a.dim;
#pragma unroll
    for (int i = 0; i < kDims; i++)
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const int d = i * 32 + result_row(j, lane);
        if (d >= a.dim) continue;
        if (a.splits > 1) {
          const float v[4] = {acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]};
          put4<float>(a.part + at.split * ((int64_t)a.batch * a.queries * a.heads * a.dim) + out + d, v);
        } else {
          const float v[4] = {acc[i][j] * a.scale, acc[i][j + 1] * a.scale, acc[i][j + 2] * a.scale, acc[i][j + 3] * a.scale};
          put4<T>((T*)a.dq + out + d, v);
        }
      }
  }
};

// -------------------------------------------------------------------- dk, dv
// fp16's power of two: a tile with a dS beyond 2^15 (the first one with any, then)
// lowers it so that the wave's largest finite one lies below 2^10, and scales what
// has been added up.  A dS is off by half a step of its own, or by 2^-34 of the largest
// one that the wave has met.  (The rows' bounds |dy| |v| + |delta| in place of a look at
// each dS are no faster, 339 and 188 us where this takes 332 and 186, and a key with
// large values lowers them for keys that hardly look at it.)
constexpr float kMostSlope = 32768.0f;

// VLDS: the block's values lie in LDS, not in fragments (head_dim 128 of 16-bit
// types, whose sums leave no registers for them).
template <typename T, int D, int QT, bool VLDS> struct AttnDkv {
  using M = Mma32<T>;
  using Frag = typename M::Frag;
  static constexpr int NW = 4, kThreads = 64 * NW, kKeys = 32 * NW;
  using Tile = RowTile<T, D, QT, NW>;
  static constexpr int kSteps = D / M::kK, kDims = D / 32;
  // two buffers of Q and dy, and of the tile's lse2 and delta (64 floats each)
  static constexpr int kStage = 2 * Tile::kPlace;
  using Values = RowTile<T, D, kKeys, NW>;                 // VLDS: the block's values stay in LDS
  static constexpr int kStats = 2 * kStage, kValues = kStats + 2 * 512;
  static constexpr int kShared = kValues + (VLDS ? Values::kBytes : 0);
  static constexpr int kBlocksPerCu = D * sizeof(T) > 256 ? 1 : 2;     // registers
  static_assert(QT <= 64, "one load brings a tile's statistics");

  static __device__ inline void run(const AttnArgs& a, char* smem) {
    const AttnPlace at(a);
    if (!at.valid) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int key = (at.tile * NW + wave) * 32 + (lane & 31);
    const bool exists = key < at.length;
    const int64_t part_size = (int64_t)a.batch * a.keys * a.kv_heads * a.dim;

    RowFrags<T, D> k, v;
    k.load(row_at<T>(a.k, at.batch, at.kv_head, exists ? key : 0), exists, a.dim, lane);
    if constexpr (!VLDS) v.load(row_at<T>(a.v, at.batch, at.kv_head, exists ? key : 0), exists, a.dim, lane);
    FragReader<T, kKeys> read_v(smem + kValues, lane);
    if (VLDS && at.tile * kKeys < at.length) {
      const int64_t pitch = a.v.row * (int64_t)sizeof(T);
      Values values;
      RowStream stream;
      stream.start(row_at<T>(a.v, at.batch, at.kv_head, 0), pitch, (int64_t)at.tile * kKeys, at.length, 0, a.dim * (int)sizeof(T));
      values.start(pitch, a.dim, wave, lane);
      values.load(stream.next(), smem + kValues, wave);
    }

    // tiles of query rows: of every query head, one after the other
    const int tiles = (a.queries + QT - 1) / QT;
    const int64_t all = (int64_t)at.tile * kKeys < at.length ? (int64_t)a.group * tiles : 0;
    const int64_t per = (all + a.splits - 1) / a.splits;
    const int64_t first = at.split * per, last = first + per < all ? first + per : all;
    const int64_t pitch_q = a.q.row * (int64_t)sizeof(T), pitch_dy = a.dy.row * (int64_t)sizeof(T);
    Tile tq, tdy;
    tq.start(pitch_q, a.dim, wave, lane);
    tdy.start(pitch_dy, a.dim, wave, lane);
    int head = at.kv_head * a.group, next = 0;          // of the tile that is issued next
    int row_now = 0;                                    // first row of the tile in work
    bool fresh = true;
    if (first < last) {
      head += (int)(first / tiles);
      next = (int)(first % tiles);
      row_now = next * QT;
    }
    const int row_bytes = a.dim * (int)sizeof(T);
    RowStream queries, grads, lse2s, deltas;
    auto issue = [&](int buf) {
      if (next == 0 || fresh) {             // a head's rows
        const int64_t row = (int64_t)next * QT, stat = ((int64_t)at.batch * a.heads + head) * a.queries;
        queries.start(row_at<T>(a.q, at.batch, head, 0), pitch_q, row, a.queries, QT, row_bytes);
        grads.start(row_at<T>(a.dy, at.batch, head, 0), pitch_dy, row, a.queries, QT, row_bytes);
        lse2s.start(a.lse2 + stat, 4, row, a.queries, QT, 4);
        deltas.start(a.delta + stat, 4, row, a.queries, QT, 4);
        fresh = false;
      }
      char* lds = smem + buf * kStage;
      tq.load(queries.next(), lds, wave);
      tdy.load(grads.next(), lds + Tile::kPlace, wave);
      const uint32_t to = (uint32_t)(uintptr_t)(RINGAR_LDS void*)smem + kStats + buf * 512;
      const u32x4 l = lse2s.next(), d = deltas.next();
      if (wave == 0) load_lds_word(lane * 4, l, to);
      else if (wave == 1) load_lds_word(lane * 4, d, to + 256);
      if (++next == tiles) {
        next = 0;
        head++;
      }
    };

    f32x16 dk[kDims], dv[kDims];
#pragma unroll
    for (int i = 0; i < kDims; i++) dk[i] = dv[i] = zero16();
    int up = kMostUp;                                   // fp16 holds dS times 2^up
    float times = exists ? power_of_two(up) * Shift<T>::kBack : 0.0f;      // (keys that do not exist: dS is 0 or NaN)
    FragReader<T, QT> read(smem, lane);
    if (first < last) issue(0);
    int buf = 0;
    for (int64_t tile = first; tile < last; tile++, buf ^= 1, read.other(kStage)) {
      wait_lds();
      block_barrier();
      if (tile + 1 < last) issue(buf ^ 1);
      const float* lse2 = (const float*)(smem + kStats + buf * 512);
      const int rows_left = a.queries - row_now;        // of the tile that exist
      row_now = row_now + QT < a.queries ? row_now + QT : 0;
#pragma unroll
      for (int b = 0; b < QT / 32; b++) {
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int i = 0; i < kSteps; i++) {
          s = M::run(read.rows(0, b * 32, i), k.f[i], s);
          if constexpr (VLDS) dp = M::run(read.rows(Tile::kPlace, b * 32, i), read_v.rows(wave * 32 * 128, 0, i), dp);
          else dp = M::run(read.rows(Tile::kPlace, b * 32, i), v.f[i], dp);
          // (not more fragments ahead than there are registers)
          if (i % 2) __builtin_amdgcn_sched_barrier(0);
        }
        float p[16], ds[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int row = b * 32 + result_row(j, lane);
          const f32x4 l = *(const f32x4*)(lse2 + row), delta = *(const f32x4*)(lse2 + 64 + row);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            p[j + e] = fast_exp2(fmaf(s[j + e], a.scale2, Shift<T>::kLog2 - l[e]));
            ds[j + e] = p[j + e] * (kScaledSlopes<T> ? (dp[j + e] - delta[e]) * times : dp[j + e] - delta[e]);
          }
        }
        if (rows_left < QT) {                 // rows past the end
#pragma unroll
          for (int j = 0; j < 16; j++)
            if (b * 32 + result_row(j, lane) >= rows_left) p[j] = ds[j] = 0.0f;
          if (b == 0 && a.dy.row < a.dim) {   // (what a wave has read of them so far it has just put away)
            Tile::clear(smem + buf * kStage + Tile::kPlace, rows_left, wave, lane);
            wait_lds();
            block_barrier();
          }
        }
        if constexpr (kScaledSlopes<T>) {
          float most = fmaxf(fabsf(ds[0]), fabsf(ds[1]));
#pragma unroll
          for (int j = 2; j < 16; j++) most = fmaxf(most, fabsf(ds[j]));
          if (__any(most > kMostSlope)) {
            most = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; j++) most = fabsf(ds[j]) < INFINITY ? fmaxf(most, fabsf(ds[j])) : most;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
            const int less = __builtin_amdgcn_readfirstlane(most > 1024.0f ? exponent_of(most) - 10 : 0);
            const float by = power_of_two(-less);
            up -= less;
            times *= by;
#pragma unroll
            for (int j = 0; j < 16; j++) ds[j] *= by;
#pragma unroll
            for (int i = 0; i < kDims; i++) dk[i] *= by;
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        constexpr int kEach = 16 / sizeof(T);
#pragma unroll
        for (int f = 0; f < 32 / M::kK; f++) {
          const Frag pf = result_frag<T>(p + f * kEach), df = result_frag<T>(ds + f * kEach);
#pragma unroll
          for (int i = 0; i < kDims; i++) {
            dv[i] = M::run(read.cols(Tile::kPlace, b * 32 + f * M::kK, i * 32), pf, dv[i]);
            dk[i] = M::run(read.cols(0, b * 32 + f * M::kK, i * 32), df, dk[i]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    }
    if (key >= a.keys) return;
    if constexpr (kScaledSlopes<T>) {
      const float down = power_of_two(-up);
#pragma unroll
      for (int i = 0; i < kDims; i++) dk[i] *= down;
    }
    const int64_t out = (((int64_t)at.batch * a.keys + key) * a.kv_heads + at.kv_head) * a.dim;
#pragma unroll
    for (int i = 0; i < kDims; i++)
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const int d = i * 32 + result_row(j, lane);
        if (d >= a.dim) continue;
        // keys past the length: zeros, whatever their columns have added up
        float vk[4], vv[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          vk[e] = exists ? dk[i][j + e] * (a.splits > 1 ? 1.0f : a.scale) : 0.0f;
          vv[e] = exists ? dv[i][j + e] * Shift<T>::kBack : 0.0f;
        }
        if (a.splits > 1) {
          put4<float>(a.part + (2 * at.split) * part_size + out + d, vk);
          put4<float>(a.part + (2 * at.split + 1) * part_size + out + d, vv);
        } else {
          if (a.dk) put4<T>((T*)a.dk + out + d, vk);
          if (a.dv) put4<T>((T*)a.dv + out + d, vv);
        }
      }
  }
};

template <typename K> __global__ __launch_bounds__(K::kThreads, K::kBlocksPerCu) void attn_dq(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[K::kShared];
  K::run(a, smem);
}
template <typename K> __global__ __launch_bounds__(K::kThreads, K::kBlocksPerCu) void attn_dkv(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[K::kShared];
  K::run(a, smem);
}

template <typename T> hipError_t attn_delta_of(const AttnArgs& a, hipStream_t st) {
  const int64_t blocks = ((int64_t)a.batch * a.heads * a.queries + 127) / 128;
  return launch_kernel(attn_delta<T>, dim3((unsigned)(blocks < most_blocks(256) ? blocks : most_blocks(256))), 256, st, a);
}

template <typename T> hipError_t attn_dq_of(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)attn_blocks(a));
  if (a.dim <= 64) return launch_kernel(attn_dq<AttnDq<T, 64>>, grid, 256, st, a);
  if constexpr (sizeof(T) == 4) {
    if (a.dim <= 96) return launch_kernel(attn_dq<AttnDq<T, 96>>, grid, 256, st, a);
  }
  return launch_kernel(attn_dq<AttnDq<T, 128>>, grid, 256, st, a);
}

template <typename T> hipError_t attn_dkv_of(const AttnArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)attn_blocks(a));
  if (a.dim <= 64) return launch_kernel(attn_dkv<AttnDkv<T, 64, 64, false>>, grid, 256, st, a);
  if constexpr (sizeof(T) == 4) {
    if (a.dim <= 96) return launch_kernel(attn_dkv<AttnDkv<T, 96, 32, false>>, grid, 256, st, a);
  }
  return launch_kernel(attn_dkv<AttnDkv<T, 128, 32, sizeof(T) == 2>>, grid, 256, st, a);
}

}  // namespace ringar
