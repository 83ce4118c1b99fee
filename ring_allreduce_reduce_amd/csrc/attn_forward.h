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
// matrix instruction's operand; l sums what was not rounded).  m is raised only where
// a row passes it by 8 (a factor of 256 in P, which fp32 sums and either type
// hold): most tiles then scale nothing.
//
// Rows in plenty: a block's 4 waves take 32 rows each and share the tiles.
// Few rows (one tile): its waves share the rows and take the tiles in turn,
// each its own from memory, joined over LDS at the end; more blocks along the
// keys where the GPU has room, joined by a second launch.
#pragma once

#include "attn_tile.h"

namespace ringar {

constexpr float kRaise = 8.0f;

// NW waves.  FEW: they share the rows and have tiles of their own.
template <typename T, int D, int KT, int NW, bool FEW> struct AttnForward {
  using M = Mma32<T>;
  using Frag = typename M::Frag;
  using Tile = RowTile<T, D, KT, FEW ? 1 : NW>;
  static constexpr int kThreads = 64 * NW;
  static constexpr int kSteps = D / M::kK, kBlocks = KT / 32, kDims = D / 32;
  static constexpr int kSets = FEW ? NW : 1;              // tiles in work at a time
  static constexpr int kShared = kSets * 4 * Tile::kBytes;
  static constexpr int kJoinRow = D + 4;                  // FEW: floats of a row, shifted over the banks
  static_assert(!FEW || kShared >= NW * 32 * (kJoinRow + 2) * 4, "the waves' sums fit");

  static __device__ inline void run(const AttnArgs& a, char* smem);
};

template <typename T, int D, int KT, int NW, bool FEW>
__device__ inline void AttnForward<T, D, KT, NW, FEW>::run(const AttnArgs& a, char* smem) {
  const AttnPlace at(a);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = at.tile * (FEW ? 32 : 32 * NW) + (FEW ? 0 : wave * 32) + (lane & 31);
  const bool exists = r < a.rows;
  const int r_in = exists ? r : a.rows - 1;
  const int head = at.head(a, r_in), query = r_in % a.queries;

  RowFrags<T, D> q;
  q.load(row_at<T>(a.q, at.batch, head, query), exists, a.dim, lane);

  // this block's tiles of keys
  const int all = (at.length + KT - 1) / KT, per = (all + a.splits - 1) / a.splits;
  const int first = at.split * per, last = first + per < all ? first + per : all;
  constexpr int kTurn = FEW ? NW : 1;
  int tile = first + (FEW ? wave : 0);

  const int64_t pitch_k = a.k.row * (int64_t)sizeof(T), pitch_v = a.v.row * (int64_t)sizeof(T);
  const char* keys = (const char*)row_at<T>(a.k, at.batch, at.kv_head, 0);
  const char* values = (const char*)row_at<T>(a.v, at.batch, at.kv_head, 0);
  Tile tk, tv;
  tk.start(pitch_k, a.dim, FEW ? 0 : wave, lane);
  tv.start(pitch_v, a.dim, FEW ? 0 : wave, lane);
  char* mine = smem + (FEW ? wave * 4 * Tile::kBytes : 0);
  auto issue = [&](int t, int buf) {
    const int64_t row = (int64_t)t * KT, left = at.length - 1 - row;
    char* lds = mine + buf * 2 * Tile::kBytes;
    tk.load(buffer_of(keys + row * pitch_k, left * pitch_k + a.dim * (int)sizeof(T)), lds, FEW ? 0 : wave);
    tv.load(buffer_of(values + row * pitch_v, left * pitch_v + a.dim * (int)sizeof(T)), lds + Tile::kBytes, FEW ? 0 : wave);
  };

  f32x16 o[kDims];
#pragma unroll
  for (int i = 0; i < kDims; i++) o[i] = zero16();
  float top = -INFINITY, sum = 0.0f;          // sum: of this lane's half of the keys

  FragReader<T, KT> read(mine, lane);
  if (tile < last) issue(tile, 0);
  for (int buf = 0; tile < last; tile += kTurn, buf ^= 1, read.other(2 * Tile::kBytes)) {
    // the tile has landed, and every wave is done with the other buffer
    wait_lds();
    if constexpr (!FEW) block_barrier();
    if (tile + kTurn < last) issue(tile + kTurn, buf ^ 1);
    f32x16 s[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; b++) {
      s[b] = zero16();
#pragma unroll
      for (int i = 0; i < kSteps; i++) s[b] = M::run(read.rows(0, b * 32, i), q.f[i], s[b]);
    }
    const int left = at.length - tile * KT;   // keys of the tile that exist
    if (left < KT) {
#pragma unroll
      for (int b = 0; b < kBlocks; b++)
#pragma unroll
        for (int i = 0; i < 16; i++)
          if (b * 32 + result_row(i, lane) >= left) s[b][i] = -INFINITY;
    }
    float most = -INFINITY;
#pragma unroll
    for (int b = 0; b < kBlocks; b++)
#pragma unroll
      for (int i = 0; i < 16; i++) most = fmaxf(most, s[b][i]);
    most = fmaxf(most, __shfl_xor(most, 32)) * a.scale2;
    if (__any(most > top + kRaise)) {
      const float raised = fmaxf(top, most), by = raised == -INFINITY ? 1.0f : fast_exp2(top - raised);
      top = raised;
      sum *= by;
#pragma unroll
      for (int i = 0; i < kDims; i++) o[i] *= by;
    }
    const float base = top == -INFINITY ? 0.0f : top;
    float p[kBlocks * 16];
#pragma unroll
    for (int b = 0; b < kBlocks; b++)
#pragma unroll
      for (int i = 0; i < 16; i++) {
        const float e = fast_exp2(fmaf(s[b][i], a.scale2, -base));
        p[b * 16 + i] = e;
        sum += e;
      }
#pragma unroll
    for (int f = 0; f < KT / M::kK; f++) {
      const Frag pf = result_frag<T>(p + f * (16 / (int)sizeof(T)));
#pragma unroll
      for (int i = 0; i < kDims; i++) o[i] = M::run(read.cols(Tile::kBytes, f * M::kK, i * 32), pf, o[i]);
    }
  }
  sum += __shfl_xor(sum, 32);

  const int64_t place = ((int64_t)at.split * a.batch + at.batch) * a.kv_heads + at.kv_head;
  // eight values a lane and 32 columns: y^T's columns are rows of y
  auto put = [&](int row, float top, float sum, auto value) {
    if (row >= a.rows) return;
    if (a.splits > 1) {
      const int64_t to = place * a.rows + row;
      if ((threadIdx.x & 63) < 32) {
        a.part_top[2 * to] = top;
        a.part_top[2 * to + 1] = sum;
      }
      value([&](int d, const float* v) { put4<float>(a.part + to * a.dim + d, v); }, 1.0f);
    } else {
      const int head = at.head(a, row), query = row % a.queries;
      if (a.lse && (threadIdx.x & 63) < 32)
        a.lse[((int64_t)at.batch * a.heads + head) * a.queries + query] = sum > 0.0f || sum != sum ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
      T* y = (T*)row_at<T>(a.y, at.batch, head, query);
      value([&](int d, const float* v) { put4<T>(y + d, v); }, sum == 0.0f ? 0.0f : 1.0f / sum);
    }
  };
  if constexpr (!FEW) {
    put(r, top, sum, [&](auto to, float by) {
#pragma unroll
      for (int i = 0; i < kDims; i++)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int d = i * 32 + result_row(j, lane);
          const float v[4] = {o[i][j] * by, o[i][j + 1] * by, o[i][j + 2] * by, o[i][j + 3] * by};
          if (d < a.dim) to(d, v);
        }
    });
  } else {
    // the waves' sums, through LDS
    wait_lds();
    block_barrier();
    float* all_o = (float*)smem;
    float* all_top = all_o + NW * 32 * kJoinRow;
    float* row_o = all_o + (wave * 32 + (lane & 31)) * kJoinRow;
#pragma unroll
    for (int i = 0; i < kDims; i++)
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const f32x4 v = {o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]};
        *(f32x4*)(row_o + i * 32 + result_row(j, lane)) = v;
      }
    if (lane < 32) {
      all_top[(wave * 32 + lane) * 2] = top;
      all_top[(wave * 32 + lane) * 2 + 1] = sum;
    }
    __syncthreads();
    // wave w finishes rows w, w + NW, .. : lanes take four values of a row each
    for (int i = wave; i < 32; i += NW) {
      float most = -INFINITY, total = 0.0f, by[NW];
#pragma unroll
      for (int w = 0; w < NW; w++) most = fmaxf(most, all_top[(w * 32 + i) * 2]);
#pragma unroll
      for (int w = 0; w < NW; w++) {
        const float t = all_top[(w * 32 + i) * 2];
        by[w] = t == -INFINITY ? 0.0f : fast_exp2(t - most);
        const float part = all_top[(w * 32 + i) * 2 + 1];
        total += t == -INFINITY ? part : part * by[w];       // (no keys: 0, or NaN to be kept)
      }
      put(at.tile * 32 + i, most, total, [&](auto to, float scale) {
        const int d = lane * 4;
        if (d >= a.dim) return;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW; w++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const float part = all_o[(w * 32 + i) * kJoinRow + d + j];
            v[j] += all_top[(w * 32 + i) * 2] == -INFINITY ? part : part * by[w];
          }
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] *= scale;
        to(d, v);
      });
    }
  }
}

template <typename K> __global__ __launch_bounds__(K::kThreads, K::kThreads == 256 && K::kShared <= 80 * 1024 ? 2 : 1) void attn_forward(AttnArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[K::kShared];
  K::run(a, smem);
}

// Rows whose keys were split: the parts' maxima and sums, then the parts.  A
// wave takes a row.
template <typename T> __global__ __launch_bounds__(256) void attn_forward_join(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.rows;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < rows; i += (int64_t)gridDim.x * 4) {
    float top = -INFINITY, sum = 0.0f;
    for (int s = 0; s < a.splits; s++) top = fmaxf(top, a.part_top[2 * (s * rows + i)]);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int d = lane * 4;
    for (int s = 0; s < a.splits; s++) {
      const float t = a.part_top[2 * (s * rows + i)], part = a.part_top[2 * (s * rows + i) + 1];
      const float by = t == -INFINITY ? 1.0f : fast_exp2(t - top);        // (no keys: zeros, or NaN to be kept)
      sum += part * by;
      if (d < a.dim) {
        const Pack<float, 4> o = load_pack<float, 4>(a.part + (s * rows + i) * a.dim + d);
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] += o.v[j] * by;
      }
    }
    const int row = (int)(i % a.rows);
    const int64_t bh = i / a.rows;
    const int64_t head = bh % a.kv_heads * a.group + row / a.queries, batch = bh / a.kv_heads, query = row % a.queries;
    if (a.lse && lane == 0)
      a.lse[(batch * a.heads + head) * a.queries + query] = sum > 0.0f || sum != sum ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
    const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] *= scale;
    if (d < a.dim) put4<T>((T*)row_at<T>(a.y, batch, head, query) + d, v);
  }
}

template <typename T> hipError_t attn_forward_of(const AttnArgs& a, hipStream_t st) {
  auto go = [&](auto k) {
    using K = decltype(k);
    return launch_kernel(attn_forward<K>, dim3((unsigned)attn_blocks(a)), K::kThreads, st, a);
  };
  constexpr int kFewWaves = sizeof(T) == 2 ? 4 : 2;
  hipError_t e;
  if (a.dim <= 64) e = a.few ? go(AttnForward<T, 64, 32, 4, true>()) : go(AttnForward<T, 64, 64, 4, false>());
  else e = a.few ? go(AttnForward<T, 128, 32, kFewWaves, true>()) : go(AttnForward<T, 128, sizeof(T) == 2 ? 64 : 32, 4, false>());
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.rows, blocks = (rows + 3) / 4;
  return launch_kernel(attn_forward_join<T>, dim3((unsigned)(blocks < most_blocks(256) ? blocks : most_blocks(256))), 256, st, a);
}

}  // namespace ringar
