// The activation's backward pass, with the column sums that become the bias
// gradient:
//   linear: dz = dy act'(z)
//   gated:  dg = dh u act'(g), du = dh act(g)
// dz is rounded to the operand type once, for the matrix products that read
// it twice; the sums are taken of the unrounded values.  Memory bound: each
// thread moves 16-byte packs of one column group down its block's rows, and
// the groups of rows leave a partial sum each (8192 x 2 * 10240 bf16 gated: 145
// us, 5.8 TB/s; 4096 x 16384 with sums: 71 us, 5.7 TB/s).
#include "block_types.h"

namespace ringar {
namespace {

// V columns a lane.  A lane whose pack would pass the last column takes the
// last V columns instead; the `skip` first of them are another lane's too:
// stored twice with the same value, counted once.
template <typename T, bool GATED, int V> __global__ __launch_bounds__(256) void dz_kernel(DzArgs a) {
  constexpr bool kFast = sizeof(T) == 2;
  // a wave takes 64 packs of columns; the block's four waves take rows in turn
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t nominal = ((int64_t)blockIdx.x * 64 + lane) * V;
  const int64_t c = nominal < a.n - V ? nominal : a.n - V;
  const int skip = (int)(nominal - c < V ? nominal - c : V);
  float s[V], su[V];
#pragma unroll
  for (int j = 0; j < V; j++) s[j] = su[j] = 0.0f;
#pragma unroll 2
  for (int64_t row = (int64_t)blockIdx.y * 4 + wave; row < a.rows; row += (int64_t)a.groups * 4) {
    Pack<T, V> dy = load_pack<T, V>((const T*)a.dy + row * a.lddy + c), g, u;
    const T* pre = (const T*)a.pre + row * a.ldp + c;
    if (GATED || a.pre) g = load_pack<T, V>(pre);
    if constexpr (GATED) u = load_pack<T, V>(pre + a.n);
    float z[V], d[V], act[V];
#pragma unroll
    for (int j = 0; j < V; j++) {
      z[j] = GATED || a.pre ? (float)g.v[j] : 0.0f;
      act[j] = 0.0f;
      d[j] = 1.0f;
    }
    if (GATED || a.pre) activate_grad_n<kFast, V>(a.act, z, act, d);
    Pack<T, V> og, ou;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const float e = (float)dy.v[j];
      if constexpr (GATED) {
        const float dg = e * (float)u.v[j] * d[j], du = e * act[j];
        s[j] += dg;
        su[j] += du;
        og.v[j] = (T)dg;
        ou.v[j] = (T)du;
      } else {
        s[j] += e * d[j];
        og.v[j] = (T)(e * d[j]);
      }
    }
    if (a.dz && skip < V) {
      T* o = (T*)a.dz + row * a.lddz + c;
      store_pack<T, V>(o, og);
      if constexpr (GATED) store_pack<T, V>(o + a.n, ou);
    }
  }
  if (!a.part && !a.sums) return;
  // Column sums: the waves' through LDS, then the block's row of parts; added
  // by the launch that follows (or final, where one block has all rows).
  constexpr int kSides = GATED ? 2 : 1;
  __shared__ float smem[4][64 * V];
  const int64_t cols = kSides * (int64_t)a.n, first = (int64_t)blockIdx.x * 64 * V;
#pragma unroll
  for (int which = 0; which < kSides; which++) {
    if (which) __syncthreads();
#pragma unroll
    for (int j = 0; j < V; j++)
      if (j >= skip) smem[wave][c - first + j] = which ? su[j] : s[j];
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * V; i += 256) {
      if (first + i >= a.n) continue;
      const float sum = (smem[0][i] + smem[1][i]) + (smem[2][i] + smem[3][i]);
      const int64_t at = (which ? a.n : 0) + first + i;
      if (a.sums) ((T*)a.sums)[at] = (T)sum;
      else a.part[blockIdx.y * cols + at] = sum;
    }
  }
}

template <typename T, int V> hipError_t launch(const DzArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(((int64_t)a.n + 64 * V - 1) / (64 * V)), a.groups);
  return a.gated ? launch_kernel(dz_kernel<T, true, V>, grid, 256, st, a) : launch_kernel(dz_kernel<T, false, V>, grid, 256, st, a);
}

template <typename T> hipError_t launch(const DzArgs& a, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  return a.n < V ? launch<T, 1>(a, st) : launch<T, V>(a, st);
}

// A copy with rows padded to 128 bytes (zeros), for loads that need them to
// start at 16-byte boundaries; both operands in one launch (333 and 2049 rows
// of 1023 fp16: 4.7 us, most of it the launch and one round trip).
template <typename T, int V> __global__ __launch_bounds__(256) void pack_rows(PackArgs both) {
  const bool second = blockIdx.x >= both.one[0].blocks;
  const PackArgs::One& a = both.one[second];
  // the block's first pack by one scalar division, the threads' in 32 bits
  const uint32_t per_row = (uint32_t)(a.ld_to / V);
  const int64_t first = (int64_t)(blockIdx.x - (second ? both.one[0].blocks : 0)) * 256;
  const int64_t first_row = first / per_row;
  const uint32_t in_row = (uint32_t)(first - first_row * per_row) + threadIdx.x;
  const int64_t row = first_row + in_row / per_row;
  if (row >= a.rows) return;
  const int64_t c = (int64_t)(in_row % per_row) * V;
  const T* from = (const T*)a.from + row * a.ld_from;
  Pack<T, V> v;
  if (c + V <= a.cols) {
    v = load_pack<T, V>(from + c);
  } else {
    // no load depends on another's condition: all are in flight together
#pragma unroll
    for (int j = 0; j < V; j++) {
      const T x = from[c + j < a.cols ? c + j : a.cols - 1];
      v.v[j] = c + j < a.cols ? x : (T)0.0f;
    }
  }
  store_pack<T, V>((T*)a.to + row * a.ld_to + c, v);
}

template <typename T> hipError_t pack(PackArgs& a, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  int64_t total = 0;
  for (PackArgs::One& o : a.one) {
    const int64_t blocks = (o.rows * (o.ld_to / V) + 255) / 256;   // few enough: plan_gemm
    total += blocks;
    o.blocks = (unsigned)blocks;
  }
  return total ? launch_kernel(pack_rows<T, V>, dim3((unsigned)total), 256, st, a) : hipSuccess;
}

// Zeros in a workspace's counters (a kernel, as every other access to them).
__global__ __launch_bounds__(256) void clear_words(uint32_t* words, unsigned count) {
  const unsigned i = blockIdx.x * 256 + threadIdx.x;
  if (i < count) words[i] = 0;
}

}  // namespace

hipError_t launch_clear(uint32_t* words, unsigned count, hipStream_t st) {
  return launch_kernel(clear_words, dim3((count + 255) / 256), 256, st, words, count);
}

// Row groups: enough blocks to fill the GPU (about 2048 with the column
// groups); a few rows stay in one, whose sums are then final.
int dz_groups(int dtype, int64_t rows, int64_t n) {
  const int64_t v = dtype == kF32 ? 4 : 8, each = 64 * (n < v ? 1 : v);
  int64_t g = 2048 / ((n + each - 1) / each);
  const int64_t most = rows <= 8 ? 1 : (rows + 3) / 4;
  if (g > most) g = most;
  return (int)(g < 1 ? 1 : g);
}

hipError_t launch_pack(int dtype, PackArgs a, hipStream_t st) {
  if (dtype == kF32) return pack<float>(a, st);
  if (dtype == kF16) return pack<_Float16>(a, st);
  return pack<__bf16>(a, st);
}

hipError_t launch_dz(int dtype, const DzArgs& a, hipStream_t st) {
  if (dtype == kF32) return launch<float>(a, st);
  if (dtype == kF16) return launch<_Float16>(a, st);
  return launch<__bf16>(a, st);
}

}  // namespace ringar
