// Cross attention, forward.
//
//   m = max_j s_j,  l = sum_j exp(s_j - m),  y = sum_j exp(s_j - m) v_j / l,
//   s = scale q k^T,  in one pass over the keys: when a tile raises m, what has
//   been added up is scaled by exp(m_old - m_new).
//
// A wave holds 32 query rows: Q in fragments, y^T in result registers, one
// row a lane, so that m, l and the scaling are single values of the lane.
// Query heads that share a key head lie behind each other in one run of rows.
// Tiles of keys and values come straight into LDS, two buffers in turn, one
// barrier a tile.  P is rounded to the operands' type before it meets v (the
// matrix instruction's operand; l sums what was not rounded).
//
// The first tile gives m.  A later one is taken at the m there is, without a
// look for its maximum: m is raised, and the tile taken again, only where a
// lane's exponentials add up to more than 2^12 (fp16: 65504; every type and the fp32
// sums hold those).  So most tiles cost an fma, an exponential, an addition and half
// a conversion a score.  And these take the vector units while the products take
// the matrix units: a wave works on three tiles at once, instruction by
// instruction, P v of tile t - 1, q k^T of tile t + 1 and the exponentials of t.
//
// A block's NQ x NK waves are NQ runs of 32 rows, which share tiles, and NK
// groups that take the tiles in turn, each from buffers of its own; the groups'
// sums meet in LDS at the end.  More blocks along the keys where the GPU has
// room, joined by a second launch.
//
// Times are medians, ranges two GPUs.  8 x 1024 x 2048, 16 heads of 128, bf16: 138
// .. 142 us (967 .. 995 TFLOP/s; a large library product reaches 1617): matrix units
// busy 59% of the cycles, vector units 49%, a clock of 1.7 .. 1.9 GHz; of 8192 x 16384, 8
// heads, 68% at head_dim 128 and 46% (vector units 66%) at 64.  32 tokens
// on up to 2048 keys each, 32 heads of 128 over 8: 47 us (4.1 TB/s; a large copy
// 5.1): memory.
#pragma once

#include "attn_tile.h"

namespace ringar {

// fp16 has steps of 2^-24 below 2^-14, and P is 2^-24 of the first tile's largest
// where a row of a hundred thousand keys looks at one of them and, together, at 1% of
// the others (as much as there is, where that one's value is zero).  So m is held 10
// below the largest score, in powers of two: P up to 2^10 then, and 2^-24 of it a normal
// number.  That leaves 2^6 for later tiles, which scores far apart would often
// pass; the first that does lifts every row of the wave by 6.  (8 x 1024 x 2048, 16 heads
// of 128, fp16, without and with this: 149 / 150 us, of queries three times as
// large 154 / 154, of six times 161 / 161.)
template <typename T> constexpr bool kHalf = sizeof(T) == 2 && !std::is_same_v<T, __bf16>;
template <typename T> constexpr float kMostSum = kHalf<T> ? 65504.0f : 4096.0f;
template <typename T> constexpr float kBelow = kHalf<T> ? 10.0f : 0.0f;
template <typename T> constexpr float kLift = kHalf<T> ? 6.0f : 0.0f;

template <typename T, int D, int KT, int NQ, int NK> struct AttnForward {
  using M = Mma32<T>;
  using Frag = typename M::Frag;
  using Tile = RowTile<T, D, KT, NQ>;
  static constexpr int kThreads = 64 * NQ * NK;
  static constexpr int kSteps = D / M::kK, kBlocks = KT / 32, kDims = D / 32;
  static constexpr int kGroup = 4 * Tile::kPlace;         // a group's buffers: two of keys, two of values
  static constexpr int kLaneSums = (kDims * 16 + 4) * 4;  // bytes of a lane's sums, its maximum and sum
  static constexpr int kJoin = (NK - 1) * NQ * 64 * kLaneSums;
  static constexpr int kShared = NK * kGroup > kJoin ? NK * kGroup : kJoin;
  static constexpr int kBlocksPerCu = kThreads <= 256 && kShared <= 80 * 1024 && D * sizeof(T) <= 384 ? 2 : 1;      // LDS, registers
  // waves that read a tile must all have it, and be done with it, together
  static __device__ inline void arrive() {
    wait_lds();
    if constexpr (NQ > 1) block_barrier();
  }

  static __device__ inline void run(const AttnArgs& a, char* smem);
};

template <typename T, int D, int KT, int NQ, int NK>
__device__ inline void AttnForward<T, D, KT, NQ, NK>::run(const AttnArgs& a, char* smem) {
  const AttnPlace at(a);
  if (!at.valid) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wq = wave % NQ, group = wave / NQ;
  const int r = (at.tile * NQ + wq) * 32 + (lane & 31);
  const bool exists = r < a.rows;
  const int r_in = exists ? r : a.rows - 1;
  const int head = at.head(a, r_in), query = r_in % a.queries;

  RowFrags<T, D> q;
  q.load(row_at<T>(a.q, at.batch, head, query), exists, a.dim, lane);

  // this block's tiles of keys, and of them this group's
  const int all = (at.length + KT - 1) / KT, per = (all + a.splits - 1) / a.splits;
  const int first = at.split * per, last = first + per < all ? first + per : all;
  const int turns = (last - first + NK - 1) / NK, mine = (last - first - group + NK - 1) / NK;

  const int64_t pitch_k = a.k.row * (int64_t)sizeof(T), pitch_v = a.v.row * (int64_t)sizeof(T);
  const int row_bytes = a.dim * (int)sizeof(T), from = (first + group) * KT;
  RowStream keys, values;
  keys.start(row_at<T>(a.k, at.batch, at.kv_head, 0), pitch_k, from, at.length, NK * KT, row_bytes);
  values.start(row_at<T>(a.v, at.batch, at.kv_head, 0), pitch_v, from, at.length, NK * KT, row_bytes);
  Tile tk, tv;
  tk.start(pitch_k, a.dim, wq, lane);
  tv.start(pitch_v, a.dim, wq, lane);
  char* buffers = smem + group * kGroup;
  // of the turns in order
  auto issue_k = [&](int turn) {
    if (turn < mine) tk.load(keys.next(), buffers + (turn & 1) * Tile::kPlace, wq);
  };
  auto issue_v = [&](int turn) {
    if (turn < mine) tv.load(values.next(), buffers + (2 + (turn & 1)) * Tile::kPlace, wq);
  };

  // fragments of keys (b: 32 of them, s: step) and of values (f: step, i: 32 columns)
  FragReader<T, KT> read(buffers, lane);
  constexpr int kAhead = 3;                   // fragments read before they are used
  constexpr int kMmaS = kBlocks * kSteps, kMmaV = KT / M::kK * kDims;
  auto key_frag = [&](int m) { return read.rows(0, m % kBlocks * 32, m / kBlocks); };
  auto value_frag = [&](int m) { return read.cols(2 * Tile::kPlace, m / kDims * M::kK, m % kDims * 32); };

  constexpr int kFrags = KT / M::kK, kValues = kBlocks * 16;      // P's fragments; a lane's scores
  f32x16 o[kDims];
#pragma unroll
  for (int i = 0; i < kDims; i++) o[i] = zero16();
  float below = kBelow<T>;
  float top = -INFINITY, sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};      // of this lane's half of the keys

  // The products of a turn, one matrix instruction after the other: P v of the
  // reader's values (0 .. kMmaV - 1), then q k^T of its keys but for the last step
  // of the contraction, which end_scores() adds.  before(), then with() after each
  // instruction, run beside them; each reads the fragment kAhead later.
  constexpr int kMma = kMmaV + kMmaS;
  Frag kf[kAhead];
  f32x16 begun[kBlocks];
  auto frag = [&](int m) { return m < kMmaV ? value_frag(m) : key_frag(m - kMmaV); };
  auto products = [&](int from, int to, const Frag* p, auto before, auto with) {
#pragma unroll
    for (int m = 0; m < kAhead; m++) kf[(from + m) % kAhead] = frag(from + m);
    before();
    if (to > kMmaV)
#pragma unroll
      for (int b = 0; b < kBlocks; b++) begun[b] = zero16();
#pragma unroll
    for (int m = from; m < to; m++) {
      if (m < kMmaV) o[m % kDims] = M::run(kf[m % kAhead], p[m / kDims], o[m % kDims]);
      else begun[(m - kMmaV) % kBlocks] = M::run(kf[m % kAhead], q.f[(m - kMmaV) / kBlocks], begun[(m - kMmaV) % kBlocks]);
      if (m + kAhead < kMma && (to > kMmaV || m + kAhead < kMmaV)) kf[m % kAhead] = frag(m + kAhead);
      with(m);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto end_scores = [&](f32x16* s) {
#pragma unroll
    for (int m = kMma - kBlocks; m < kMma; m++)
      s[(m - kMmaV) % kBlocks] = M::run(kf[m % kAhead], q.f[(m - kMmaV) / kBlocks], begun[(m - kMmaV) % kBlocks]);
  };
  // the i-th of a lane's scores: its exponential into P's fragments and a sum
  auto exponential = [&](const f32x16* s, Frag* p, float* sum, int i) {
    constexpr int kEach = 16 / sizeof(T);
    const float e = fast_exp2(fmaf(s[i / 16][i % 16], a.scale2, -top));
    sum[i & 3] += e;
    p[i / kEach][i % kEach] = (T)e;
    // (converted here, not where it is used: half the registers)
    if (i % kEach == kEach - 1) asm volatile("" : "+v"(p[i / kEach]));
  };
  // a tile taken with a look for its maximum, m raised by `lift` at least; `left` of its keys exist
  auto raise = [&](f32x16* s, Frag* p, int left, float lift = 0.0f) {
    if (left < KT) {
#pragma unroll
      for (int b = 0; b < kBlocks; b++)
#pragma unroll
        for (int i = 0; i < 16; i++)
          if (b * 32 + result_row(i, lane) >= left) s[b][i] = -INFINITY;
    }
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < kValues; i++) most = fmaxf(most, s[i / 16][i % 16]);
    most = fmaxf(most, __shfl_xor(most, 32)) * a.scale2 - below;
    const float raised = fmaxf(top + lift, most), by = raised == -INFINITY ? 1.0f : fast_exp2(top - raised);
    top = raised == -INFINITY ? -3e38f : raised;      // (no finite score yet: the first one passes any m of use)
#pragma unroll
    for (int i = 0; i < 4; i++) sums[i] *= by;
#pragma unroll
    for (int i = 0; i < kDims; i++) o[i] *= by;
#pragma unroll
    for (int i = 0; i < kValues; i++) exponential(s, p, sums, i);
  };

  constexpr auto kBefore = [] {};
  constexpr auto kNothing = [](int) {};
  auto only_scores = [&] { products(kMmaV, kMma - kBlocks, nullptr, kBefore, kNothing); };
  const int left = at.length - from - (mine - 1) * NK * KT;       // keys of the last tile
  // Turns between the first and the last, and the last where it is whole, are
  // the loop's; what is rare in them leaves it, or the compiler would keep a
  // second place for all sums.
  const int whole = left < KT ? mine - 1 : mine;
  f32x16 s[kBlocks];
  Frag p[kFrags];
  issue_k(0);
  issue_k(1);
  issue_v(0);
  // the first keys; what follows them may still be on its way
  if (mine > 1) wait_lds<2 * Tile::kLoads>();
  else wait_lds<Tile::kLoads>();
  if constexpr (NQ > 1) block_barrier();
  if (mine > 0) {
    only_scores();
    end_scores(s);
    raise(s, p, mine == 1 ? left : KT);
  }
  // A turn's start: the next tile's keys and the last one's values have landed,
  // and every wave is done with what lies in the other buffers.
  auto start = [&](int turn) {
    arrive();
    issue_k(turn + 2);
    if (turn > 0) issue_v(turn);
    read.other(Tile::kPlace);
  };
  if (turns > 0) {
    start(0);
    if (mine > 1) {
      only_scores();
      end_scores(s);
    }
    for (int turn = 1; turn < whole; turn++) {
      bool over = false;
      float part[4];
      Frag p_next[kFrags];
      for (; turn < whole; turn++) {
        start(turn);
        // The exponentials, evenly, up to the last of the scores, which then
        // need no second place.
        constexpr int kFirst = kValues / 8;
#pragma unroll
        for (int i = 0; i < 4; i++) part[i] = 0.0f;
        products(0, kMma - kBlocks, p,        // (after the last tile: scores of what lies there, not used)
                 [&] {
#pragma unroll
                   for (int i = 0; i < kFirst; i++) exponential(s, p_next, part, i);
                 },
                 [&](int m) {
#pragma unroll
                   for (int i = kFirst; i < kValues; i++)
                     if ((i - kFirst) * (kMma - kBlocks) / (kValues - kFirst) == m) exponential(s, p_next, part, i);
                 });
#pragma unroll
        for (int f = 0; f < kFrags; f++) p[f] = p_next[f];
        over = __any((part[0] + part[1]) + (part[2] + part[3]) > kMostSum<T>);
        if (over) break;
#pragma unroll
        for (int i = 0; i < 4; i++) sums[i] += part[i];
        end_scores(s);
      }
      if (!over) break;
      const float lift = below > kBelow<T> - kLift<T> ? kLift<T> : 0.0f;
      below -= lift;
      raise(s, p, KT, lift);
      end_scores(s);
    }
    if (mine > 1 && whole < mine) {           // the last tile, with keys that do not exist
      start(whole);
      products(0, kMmaV, p, kBefore, kNothing);
      raise(s, p, left);
    }
    // the last tile's values (a group whose last turn is missing keeps the others company)
    if (NQ > 1 && NK > 1 && mine > 0 && mine < turns) arrive();
    arrive();
    read.other(Tile::kPlace);
    if (pitch_v < row_bytes) {
      if (mine > 0 && left < KT) Tile::clear(buffers + (2 + ((mine - 1) & 1)) * Tile::kPlace, left, wq, lane);
      arrive();
    }
    if (mine > 0) products(0, kMmaV, p, kBefore, kNothing);
  }
  float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  sum += __shfl_xor(sum, 32);
  if (sum == 0.0f) top = -INFINITY;

  if constexpr (NK > 1) {
    // the groups' sums, through LDS, a lane's own values at a time
    arrive();
    block_barrier();
    typedef float f32x4_lds __attribute__((ext_vector_type(4)));
    auto slot = [&](int g, int i) { return (f32x4_lds*)(smem + (((g - 1) * NQ + wq) * (kDims * 4 + 1) + i) * 1024) + lane; };
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < kDims; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) *slot(group, i * 4 + j) = f32x4_lds{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
      *slot(group, kDims * 4) = f32x4_lds{top, sum, 0.0f, 0.0f};
    }
    __syncthreads();
    if (group > 0) return;
    float tops[NK], most = top, total = 0.0f;
    tops[0] = top;
#pragma unroll
    for (int g = 1; g < NK; g++) {
      tops[g] = (*slot(g, kDims * 4))[0];
      most = fmaxf(most, tops[g]);
    }
    // a group that saw no finite score: zeros, or NaN to be kept
    auto by = [&](int g) { return tops[g] == -INFINITY ? 1.0f : fast_exp2(tops[g] - most); };
    total = sum * by(0);
#pragma unroll
    for (int i = 0; i < kDims; i++) o[i] *= by(0);
#pragma unroll
    for (int g = 1; g < NK; g++) {
      total += (*slot(g, kDims * 4))[1] * by(g);
#pragma unroll
      for (int i = 0; i < kDims; i++)
#pragma unroll
        for (int j = 0; j < 16; j++) o[i][j] = fmaf((*slot(g, i * 4 + j / 4))[j % 4], by(g), o[i][j]);
    }
    top = most;
    sum = total;
  }
  if (!exists) return;
  const int64_t part = (((int64_t)at.split * a.batch + at.batch) * a.kv_heads + at.kv_head) * a.rows + r;
  if (lane < 32) {
    if (a.splits > 1) {
      a.part_top[2 * part] = top;
      a.part_top[2 * part + 1] = sum;
    } else if (a.lse) {
      a.lse[((int64_t)at.batch * a.heads + head) * a.queries + query] =
          sum > 0.0f || sum != sum ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
    }
  }
  const float by = a.splits > 1 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
  T* y = (T*)row_at<T>(a.y, at.batch, head, query);
#pragma unroll
  for (int i = 0; i < kDims; i++)
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const int d = i * 32 + result_row(j, lane);
      const float v[4] = {o[i][j] * by, o[i][j + 1] * by, o[i][j + 2] * by, o[i][j + 3] * by};
      if (d >= a.dim) continue;
      if (a.splits > 1) put4<float>(a.part + part * a.dim + d, v);
      else put4<T>(y + d, v);
    }
}

template <typename K> __global__ __launch_bounds__(K::kThreads, K::kBlocksPerCu * K::kThreads / 256) void attn_forward(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[K::kShared];
  K::run(a, smem);
}

// Rows whose keys were split: the parts in order, four values of a row a thread.
template <typename T> __global__ __launch_bounds__(256) void attn_forward_join(AttnArgs a) {
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.rows;
  const int quads = a.dim / 4;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < rows * quads; at += (int64_t)gridDim.x * 256) {
    const int64_t i = at / quads;
    const int d = (int)(at % quads) * 4;
    float top = -INFINITY, sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.splits; s++) top = fmaxf(top, a.part_top[2 * (s * rows + i)]);
    for (int s = 0; s < a.splits; s++) {
      const float t = a.part_top[2 * (s * rows + i)], part = a.part_top[2 * (s * rows + i) + 1];
      const float by = t == -INFINITY ? 1.0f : fast_exp2(t - top);        // (no keys: zeros, or NaN to be kept)
      sum = fmaf(part, by, sum);
      const Pack<float, 4> o = load_pack<float, 4>(a.part + (s * rows + i) * a.dim + d);
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] = fmaf(o.v[j], by, v[j]);
    }
    const int row = (int)(i % a.rows);
    const int64_t bh = i / a.rows;
    const int64_t head = bh % a.kv_heads * a.group + row / a.queries, batch = bh / a.kv_heads, query = row % a.queries;
    if (a.lse && d == 0)
      a.lse[(batch * a.heads + head) * a.queries + query] = sum > 0.0f || sum != sum ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
    const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] *= scale;
    put4<T>((T*)row_at<T>(a.y, batch, head, query) + d, v);
  }
}

template <typename T> hipError_t attn_forward_of(const AttnArgs& a, hipStream_t st) {
  auto go = [&](auto k) {
    using K = decltype(k);
    return launch_kernel(attn_forward<K>, dim3((unsigned)attn_blocks(a)), K::kThreads, st, a);
  };
  constexpr bool kWide = sizeof(T) == 4;
  hipError_t e = hipSuccess;
  // (fp32 beyond 64: no registers for eight waves, LDS for two of few rows')
  if (a.dim <= 64) {
    if (a.form == kManyRows) e = go(AttnForward<T, 64, kWide ? 32 : 64, 4, 1>());
    else if (a.form == kSomeRows) e = go(AttnForward<T, 64, kWide ? 32 : 64, 4, 2>());
    else e = go(AttnForward<T, 64, 32, 1, 4>());
  } else if constexpr (kWide) {
    if (a.dim <= 96) e = a.form == kManyRows ? go(AttnForward<T, 96, 32, 4, 1>()) : go(AttnForward<T, 96, 32, 1, 2>());
    else e = a.form == kManyRows ? go(AttnForward<T, 128, 32, 4, 1>()) : go(AttnForward<T, 128, 32, 1, 2>());
  } else {
    if (a.form == kManyRows) e = go(AttnForward<T, 128, 64, 4, 1>());
    else if (a.form == kSomeRows) e = go(AttnForward<T, 128, 64, 4, 2>());
    else e = go(AttnForward<T, 128, 32, 1, 4>());
  }
  if (e != hipSuccess || a.splits == 1) return e;
  // four values a thread
  const int64_t threads = (int64_t)a.batch * a.kv_heads * a.rows * (a.dim / 4), blocks = (threads + 255) / 256;
  return launch_kernel(attn_forward_join<T>, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), 256, st, a);
}

}  // namespace ringar
