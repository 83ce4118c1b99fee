// The backward pass of a few rows (single tokens): all three gradients in one
// pass over the weight.
//
//   dz = dy act'(z) (gated: [dy u act'(g), dy act(g)]);
//   dx = dz W,  dW = dz^T x,  db = sum_rows dz
//
// With so few rows the products are memory bound: W is read once, dW written
// once, and everything else is small.  A block takes some rows of W (n) and
// 64 packs of columns (fewer for a narrow W), four rows or more at a time; its dz sits in LDS, x and the sums of dx in registers, and every
// row costs one 16-byte load, one 16-byte store and 2 M fused multiply-adds a
// value.  The blocks' parts of dx are added, in order, by a second pass (a last
// block to arrive took 10 us for what that pass does in 3).
#include "block_types.h"

namespace ringar {
namespace {

constexpr int kMostN = 128;            // rows of W a block takes at most

template <typename T, int V, int M> __global__ __launch_bounds__(256) void few_backward(FewArgs a) {
  constexpr bool kFast = sizeof(T) == 2;
  __shared__ float dz[M][kMostN];
  __shared__ float lds[256 * (V + 1)];
  const int n0 = blockIdx.y * a.n_each;
  const int count = a.wide - n0 < a.n_each ? a.wide - n0 : a.n_each;
  // dz of the block's rows of W; it feeds fp32 multiply-adds and stays as it is
  for (int i = threadIdx.x; i < count; i += 256) {
    const int col = n0 + i, at = a.gated && col >= a.n ? col - a.n : col;
    float sum = 0.0f;
#pragma unroll
    for (int m = 0; m < M; m++) {
      float v = 0.0f;
      if (m < a.rows) {
        v = (float)((const T*)a.dy)[m * a.lddy + at];
        if (a.pre) {
          const T* pre = (const T*)a.pre + m * a.ldp;
          float act, d;
          activate_grad<kFast>(a.act, (float)pre[at], &act, &d);
          v *= !a.gated ? d : col < a.n ? (float)pre[a.n + at] * d : act;
        }
      }
      sum += v;
      dz[m][i] = v;
    }
    if (a.db && blockIdx.x == 0) ((T*)a.db)[col] = (T)sum;
  }
  __syncthreads();
  if (!a.dx && !a.dw) return;

  // thread: pack `kt` of the block's columns, rows of W nt, nt + rows_at_once, ...
  const int across = 1 << a.across_log, kt = threadIdx.x & (across - 1), nt = threadIdx.x >> a.across_log;
  const int rows_at_once = 256 >> a.across_log;
  const int64_t nominal = ((int64_t)blockIdx.x * across + kt) * V;
  const int64_t c = nominal < a.k - V ? nominal : a.k - V;       // the last packs overlap: the same values twice
  const bool mine = nominal < a.k;
  float x[M][V], acc[M][V];
#pragma unroll
  for (int m = 0; m < M; m++) {
    Pack<T, V> p = {};
    if (a.dw) p = load_pack<T, V>((const T*)a.x + (m < a.rows ? m : 0) * a.ldx + c);
#pragma unroll
    for (int j = 0; j < V; j++) {
      x[m][j] = m < a.rows ? (float)p.v[j] : 0.0f;
      acc[m][j] = 0.0f;
    }
  }
  auto turn = [&](int i, const Pack<T, V>& w) {
    float z[M];
#pragma unroll
    for (int m = 0; m < M; m++) z[m] = dz[m][i];
    if (a.dx) {
#pragma unroll
      for (int j = 0; j < V; j++) {
        const float v = (float)w.v[j];
#pragma unroll
        for (int m = 0; m < M; m++) acc[m][j] = fmaf(z[m], v, acc[m][j]);
      }
    }
    if (a.dw && mine) {
      Pack<T, V> o;
#pragma unroll
      for (int j = 0; j < V; j++) {
        float s = 0.0f;
#pragma unroll
        for (int m = 0; m < M; m++) s = fmaf(z[m], x[m][j], s);
        o.v[j] = (T)s;
      }
      store_pack<T, V>((T*)a.dw + (n0 + i) * a.lddw + c, o);
    }
  };
  constexpr int U = 4;                 // rows of W in flight
  Pack<T, V> w[U];
  auto fetch = [&](int i) {
    return load_pack<T, V>((const T*)a.w + (int64_t)(n0 + (i < count ? i : count - 1)) * a.ldw + c);
  };
  if (a.dx)
#pragma unroll
    for (int u = 0; u < U; u++) w[u] = fetch(nt + u * rows_at_once);
  for (int i = nt; i < count; i += U * rows_at_once) {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int at = i + u * rows_at_once;
      const Pack<T, V> now = w[u];
      if (a.dx) w[u] = fetch(at + U * rows_at_once);
      if (at < count) turn(at, now);
    }
  }
  if (!a.dx) return;

  // The sums of a column over the block's threads, through LDS so that the
  // stores run along the columns; then over the blocks.
  const int64_t first = (int64_t)blockIdx.x * across * V;
  const int width = (int)(a.k - first < across * V ? a.k - first : across * V);
#pragma unroll
  for (int m = 0; m < M; m++) {
    if (m >= a.rows) break;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; j++) lds[threadIdx.x * (V + 1) + j] = acc[m][j];
    __syncthreads();
    for (int i = threadIdx.x; i < width; i += 256) {
      // where the pack of this column starts, and so its place in it
      const int64_t at = first + i / V * V;
      const int j = i % V + (at > a.k - V ? (int)(at - (a.k - V)) : 0);
      float s = 0.0f;
      for (int r = 0; r < rows_at_once; r++) s += lds[(r * across + i / V) * (V + 1) + j];
      if (a.parts == 1) ((T*)a.dx)[m * a.lddx + first + i] = (T)s;
      else a.part[((int64_t)blockIdx.y * a.rows + m) * a.k + first + i] = s;
    }
  }
}

// 64 values of dx a block; its waves take the parts in turn (one thread for
// all 412 parts of 4 x 117: 11 us), then the waves' sums in order.
template <typename T> __global__ __launch_bounds__(1024) void few_join(FewArgs a) {
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t width = (int64_t)a.rows * a.k, i = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (i < width) s = sum_parts<8>(w, 16, a.parts, [&](int p) { return a.part[p * width + i]; });
  lds[w][lane] = s;
  __syncthreads();
  if (w || i >= width) return;
  s = 0.0f;
#pragma unroll
  for (int p = 0; p < 16; p++) s += lds[p][lane];
  ((T*)a.dx)[i / a.k * a.lddx + i % a.k] = (T)s;
}

template <typename T, int V, int M> hipError_t launch(const FewArgs& a, hipStream_t st) {
  const int64_t packs = (a.k + V - 1) / V;
  const hipError_t e = launch_kernel(few_backward<T, V, M>, dim3((unsigned)((packs + (1 << a.across_log) - 1) >> a.across_log), a.parts), 256, st, a);
  if (e != hipSuccess || !a.dx || a.parts == 1) return e;
  return launch_kernel(few_join<T>, dim3((unsigned)(((int64_t)a.rows * a.k + 63) / 64)), 1024, st, a);
}

}  // namespace

// Where the one pass wins over the products of the matrix kernels.  Its
// multiply-adds are 2 a row and value on the vector units, so rows end it.  us
// of the call, one pass and products:
//   4096 x 4096 bf16, 1, 2, 4 rows: 15.8, 17.8, 22.5 and 28.1, 28.1, 28.4 (8
//     rows: 33 and 31); fp32, 1, 4, 8 rows: 30.6, 33.3, 38.2 and 50.6, 50.7, 51.5;
//   4096 in, 16384 out, bf16, 1 and 4 rows: 50.7, 57.2 and 74.9, 75.0;
//   small weights with dx: 512 x 512 bf16 7.1, 8.2, 11.0 and 8.0, 8.0, 8.1 (its
//     second launch waits for the first); 8 rows of fp32 11.9 and 10.7;
//   without dx one launch: 512 x 512 bf16, 1 and 4 rows 3.4, 4.9 and 6.6, 6.9.
// The launch that adds the parts takes a block for every 64 values of dx.
bool few_rows(int dtype, int64_t rows, int64_t wide, int64_t k) {
  return (rows * k + 63) / 64 <= most_blocks(1024) && rows >= 1 && rows <= (dtype == kF32 ? 8 : 4) && k >= 8 && wide >= 1 && wide <= 65535ll * kMostN;
}

// Columns across, rows of W a block, parts of dx.
size_t plan_few(int dtype, FewArgs& a) {
  const int v = dtype == kF32 ? 4 : 8;
  const int64_t packs = (a.k + v - 1) / v;
  a.across_log = 0;
  while (a.across_log < 6 && (1 << a.across_log) < packs) a.across_log++;
  const int64_t columns = (packs + (1 << a.across_log) - 1) >> a.across_log;
  const int at_once = 256 >> a.across_log;
  // about 1024 blocks, with four turns or more each
  int64_t each = (a.wide * columns + 1023) / 1024;
  if (each < 4 * at_once) each = 4 * at_once;
  if (each > kMostN || (a.wide + each - 1) / each > 65535) each = kMostN;
  a.n_each = (int)each;
  a.parts = (int)((a.wide + each - 1) / each);
  return a.dx && a.parts > 1 ? (size_t)a.parts * a.rows * a.k * 4 : 0;
}

hipError_t launch_few(int dtype, const FewArgs& a, hipStream_t st) {
  if (dtype == kF32) return a.rows <= 2 ? launch<float, 4, 2>(a, st) : a.rows <= 4 ? launch<float, 4, 4>(a, st) : launch<float, 4, 8>(a, st);
  if (dtype == kF16) return a.rows <= 2 ? launch<_Float16, 8, 2>(a, st) : launch<_Float16, 8, 4>(a, st);
  return a.rows <= 2 ? launch<__bf16, 8, 2>(a, st) : launch<__bf16, 8, 4>(a, st);
}

}  // namespace ringar
