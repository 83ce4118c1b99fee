// Layer norm, forward and backward, and the column sums that finish the
// parameter gradients.
//
//   h = (x - mu) r,  r = 1 / sqrt(var + eps),  y = h w + b
//   g = dy w,  dx = r (g - mean(g) - h mean(g h)),  dw = sum dy h,  db = sum dy
//
// A row is held in the registers of TPR threads (E elements each) between
// its statistics and its output, so memory sees each input and output once;
// the statistics are two passes over those registers (mean, then the centred
// square), in fp32.  The backward pass gives each thread the same columns of
// every row it meets: the parameter gradients build up in registers, leave
// as one partial row per block, and are added in block order by a second
// kernel (no atomics: results do not depend on scheduling).
//
// Memory bound: forward 16384 x 8192 bf16 92 us (5.8 TB/s), backward 16384 x
// 4096 bf16 73 us and 5 us of column sums (5.5 TB/s).
#include "block_types.h"

namespace ringar {
namespace {

constexpr int kBlock = 256;

// Sum of `v` over the TPR threads that share a row.
template <int TPR> __device__ inline float row_sum(float v, float* smem) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) smem[wave] = v;
    __syncthreads();
    const float* row = smem + wave / (TPR / 64) * (TPR / 64);
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) v += row[i];
    __syncthreads();
  }
  return v;
}

template <int TPR> __device__ inline void row_sum2(float& u, float& v, float* smem) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o > 0; o >>= 1) {
    u += __shfl_xor(u, o);
    v += __shfl_xor(v, o);
  }
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      smem[2 * wave] = u;
      smem[2 * wave + 1] = v;
    }
    __syncthreads();
    const float* row = smem + wave / (TPR / 64) * (TPR / 64) * 2;
    u = v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) {
      u += row[2 * i];
      v += row[2 * i + 1];
    }
    __syncthreads();
  }
}

// E elements of a row: thread t of TPR holds the packs of V elements that
// start at (i * TPR + t) * V.  A pack that would pass the row's end starts V
// before the end instead, and its first `skip` elements, which belong to
// other packs, are held as zeros and not stored: loads never branch, so all
// of them are in flight together, at any width of at least V.
template <typename T, int TPR, int E, int V> struct Row {
  static constexpr int P = E / V;
  int col[P], skip[P];

  __device__ inline Row(int cols, int t) {
#pragma unroll
    for (int i = 0; i < P; i++) {
      const int c = (i * TPR + t) * V;
      col[i] = c < cols - V ? c : cols - V;
      skip[i] = c - col[i];
    }
  }
  // the row as it lies in memory
  template <typename U> struct Raw {
    Pack<U, V> q[P];
  };
  template <typename U> __device__ inline void load(const U* p, Raw<U>& r) const {
#pragma unroll
    for (int i = 0; i < P; i++) r.q[i] = load_pack<U, V>(p + col[i]);
  }
  template <typename U> __device__ inline void widen(const Raw<U>& r, float* out) const {
#pragma unroll
    for (int i = 0; i < P; i++)
#pragma unroll
      for (int j = 0; j < V; j++) out[i * V + j] = (float)r.q[i].v[j];
    clear(out);
  }
  __device__ inline void clear(float* v) const {
#pragma unroll
    for (int i = 0; i < P; i++)
      if (skip[i] > 0)
#pragma unroll
        for (int j = 0; j < V; j++)
          if (j < skip[i]) v[i * V + j] = 0.0f;
  }
  template <typename F> __device__ inline void each(F f) const {
#pragma unroll
    for (int i = 0; i < P; i++)
#pragma unroll
      for (int j = 0; j < V; j++)
        if (j >= skip[i]) f(i * V + j, col[i] + j);
  }
  // fp32 sums, 16 bytes at a time (value by value the partial rows of 8192 x
  // 8192 bf16 cost 10 us more: 83, not 73)
  __device__ inline void sums(float* p, const float* in) const {
    constexpr int S = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < P; i++)
#pragma unroll
      for (int h = 0; h < V; h += S) {
        if (skip[i] <= h) {
          Pack<float, S> q;
#pragma unroll
          for (int j = 0; j < S; j++) q.v[j] = in[i * V + h + j];
          store_pack<float, S>(p + col[i] + h, q);
        } else {
#pragma unroll
          for (int j = 0; j < S; j++)
            if (h + j >= skip[i]) p[col[i] + h + j] = in[i * V + h + j];
        }
      }
  }
  template <bool STREAM> __device__ inline void store(T* p, const float* in) const {
#pragma unroll
    for (int i = 0; i < P; i++) {
      if (skip[i] == 0) {
        Pack<T, V> q;
#pragma unroll
        for (int j = 0; j < V; j++) q.v[j] = (T)in[i * V + j];
        if constexpr (STREAM) stream_pack<T, V>(p + col[i], q);
        else store_pack<T, V>(p + col[i], q);
      } else {
#pragma unroll
        for (int j = 0; j < V; j++)
          if (j >= skip[i]) p[col[i] + j] = (T)in[i * V + j];
      }
    }
  }
};

template <typename T, typename W, int TPR, int E, int V, bool STREAM>
__global__ __launch_bounds__(TPR < kBlock ? kBlock : TPR) void norm_forward(NormArgs a) {
  using R = Row<T, TPR, E, V>;
  constexpr int kThreads = TPR < kBlock ? kBlock : TPR;
  constexpr int kRows = kThreads / TPR;
  __shared__ float smem[kThreads / 64];
  const int t = threadIdx.x % TPR;
  const R r(a.cols, t);
  // A block takes rows in turn: the parameters stay in its registers (as they
  // lie in memory), and the next row is on its way while this one is worked
  // on.  Every thread runs the same number of turns; a row past the end is
  // the last one again and not stored.
  const int64_t stride = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  typename R::template Raw<T> next;
  typename R::template Raw<W> w, b;
  auto fetch = [&](int64_t i) { r.template load<T>((const T*)a.x + (i < a.rows ? i : a.rows - 1) * a.ldx, next); };
  fetch(row);
  if (a.weight) r.template load<W>((const W*)a.weight, w);
  if (a.bias) r.template load<W>((const W*)a.bias, b);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride, row += stride) {
    float v[E];
    r.template widen<T>(next, v);
    fetch(row + stride);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i++) s += v[i];
    const float mean = row_sum<TPR>(s, smem) * a.inv_cols;
#pragma unroll
    for (int i = 0; i < E; i++) v[i] -= mean;
    r.clear(v);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i++) s = fmaf(v[i], v[i], s);
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, smem) * a.inv_cols + a.eps);
    if (row >= a.rows) continue;
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < E; i++) {
      const float scale = a.weight ? (float)w.q[i / V].v[i % V] : 1.0f, shift = a.bias ? (float)b.q[i / V].v[i % V] : 0.0f;
      v[i] = fmaf(v[i] * rstd, scale, shift);
    }
    r.template store<STREAM>((T*)a.y + row * a.ldy, v);
  }
}

// Rows too long for the registers: three passes, the later two from cache,
// value by value (512 x 32768: fp32 42 us, 3.2 TB/s, bf16 50, 1.3; backward 75
// and 67).
template <typename T, typename W> __global__ __launch_bounds__(1024) void norm_forward_long(NormArgs a) {
  __shared__ float smem[16];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) s += (float)x[c];
    const float mean = row_sum<1024>(s, smem) * a.inv_cols;
    s = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float e = (float)x[c] - mean;
      s = fmaf(e, e, s);
    }
    const float rstd = 1.0f / sqrtf(row_sum<1024>(s, smem) * a.inv_cols + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = (T*)a.y + row * a.ldy;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float w = a.weight ? (float)((const W*)a.weight)[c] : 1.0f;
      const float b = a.bias ? (float)((const W*)a.bias)[c] : 0.0f;
      y[c] = (T)fmaf(((float)x[c] - mean) * rstd, w, b);
    }
  }
}

template <typename T, typename W, int TPR, int E, int V, int kRows, bool STREAM>
__global__ __launch_bounds__(TPR * kRows) void norm_backward(NormArgs a) {
  using R = Row<T, TPR, E, V>;
  constexpr int kThreads = TPR * kRows;
  // A row of 32 values a thread leaves no registers for the next one (kept
  // ahead, 4096 x 16384 fp32 spilled 70 of them: 328 us, not 170).
  constexpr bool kAhead = E < 32;
  __shared__ float smem[kThreads / 64 * 2];
  const int t = threadIdx.x % TPR;
  const int lane_row = threadIdx.x / TPR;
  const R r(a.cols, t);
  // The next row is loaded while this one is worked on (kAhead).  Every thread
  // of a block runs the same number of turns; a row past the end is the last
  // one again, not counted and not stored.
  const int64_t stride = (int64_t)a.groups * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + lane_row;
  typename R::template Raw<T> rx, rdy;
  float next_mean, next_rstd;
  auto fetch = [&](int64_t i) {
    i = i < a.rows ? i : a.rows - 1;
    r.template load<T>((const T*)a.x + i * a.ldx, rx);
    r.template load<T>((const T*)a.dy + i * a.lddy, rdy);
    next_mean = a.mean[i];
    next_rstd = a.rstd[i];
  };
  if (kAhead) fetch(row);
  float dw[E], db[E];
  typename R::template Raw<W> wt;
  if (a.weight) r.template load<W>((const W*)a.weight, wt);
  auto weight = [&](int i) { return a.weight ? (float)wt.q[i / V].v[i % V] : 1.0f; };
#pragma unroll
  for (int i = 0; i < E; i++) dw[i] = db[i] = 0.0f;
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride, row += stride) {
    const bool live = row < a.rows;
    if (!kAhead) fetch(row);
    float h[E], dy[E];
    r.template widen<T>(rx, h);
    r.template widen<T>(rdy, dy);
    const float mean = next_mean, rstd = next_rstd;
    if (kAhead) fetch(row + stride);
    float sg = 0.0f, sgh = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i++) {
      dy[i] = live ? dy[i] : 0.0f;
      h[i] = (h[i] - mean) * rstd;
      dw[i] = fmaf(dy[i], h[i], dw[i]);      // dy is 0 where a pack holds no element
      db[i] += dy[i];
      dy[i] *= weight(i);
      sg += dy[i];
      sgh = fmaf(dy[i], h[i], sgh);
    }
    if (a.y) {
      row_sum2<TPR>(sg, sgh, smem);
      sg *= a.inv_cols;
      sgh *= a.inv_cols;
#pragma unroll
      for (int i = 0; i < E; i++) dy[i] = rstd * (dy[i] - sg - h[i] * sgh);
      if (live) r.template store<STREAM>((T*)a.y + row * a.ldy, dy);
    }
  }
  if (!a.part && !a.dweight && !a.dbias) return;
  // the block's rows into one partial row, or where it has them all into the gradients
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  auto put = [&](int which, int c, float s) {
    W* g = (W*)(which ? a.dbias : a.dweight);
    if (a.part) out[which * a.cols + c] = s;
    else if (g) g[c] = (W)s;
  };
  if constexpr (kRows > 1) {
    __shared__ float rows[kRows][TPR * E];
#pragma unroll
    for (int which = 0; which < 2; which++) {
      if (which) __syncthreads();
      r.sums(rows[lane_row], which ? db : dw);
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += kThreads) {
        float s = 0.0f;
#pragma unroll 4
        for (int i = 0; i < kRows; i++) s += rows[i][c];
        put(which, c, s);
      }
    }
  } else {
    if (a.part) {
      r.sums(out, dw);
      r.sums(out + a.cols, db);
    } else {
      r.each([&](int i, int c) {
        put(0, c, dw[i]);
        put(1, c, db[i]);
      });
    }
  }
}

// dx of rows too long for the registers
template <typename T, typename W> __global__ __launch_bounds__(1024) void norm_backward_long(NormArgs a) {
  __shared__ float smem[32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* dy = (const T*)a.dy + row * a.lddy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float sg = 0.0f, sgh = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float g = (float)dy[c] * (a.weight ? (float)((const W*)a.weight)[c] : 1.0f);
      sg += g;
      sgh = fmaf(g, ((float)x[c] - mean) * rstd, sgh);
    }
    row_sum2<1024>(sg, sgh, smem);
    sg *= a.inv_cols;
    sgh *= a.inv_cols;
    T* dx = (T*)a.y + row * a.ldy;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float g = (float)dy[c] * (a.weight ? (float)((const W*)a.weight)[c] : 1.0f);
      dx[c] = (T)(rstd * (g - sg - (((float)x[c] - mean) * rstd) * sgh));
    }
  }
}

// parameter gradients of such rows: one column a thread, the block's rows in
// turn
template <typename T> __global__ __launch_bounds__(256) void norm_params_long(NormArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += a.groups) {
    const float g = (float)((const T*)a.dy)[row * a.lddy + c];
    dw = fmaf(g, ((float)((const T*)a.x)[row * a.ldx + c] - a.mean[row]) * a.rstd[row], dw);
    db += g;
  }
  a.part[(int64_t)blockIdx.y * 2 * a.cols + c] = dw;
  a.part[((int64_t)blockIdx.y * 2 + 1) * a.cols + c] = db;
}

template <typename O> __global__ __launch_bounds__(1024) void col_sum(ColSumArgs a) {
  __shared__ float smem[16 * 64];
  for (unsigned block = blockIdx.x; (int64_t)block * 64 < a.width; block += gridDim.x) {
    if (block != blockIdx.x) __syncthreads();
    col_sum_block<O>(a, block, 16, smem);
  }
}

// Blocks of a kernel that loops over what it has too few of.
unsigned capped(int64_t blocks, int threads) { return (unsigned)(blocks < most_blocks(threads) ? blocks : most_blocks(threads)); }

// Threads and elements per thread of a row: the smallest shape that holds it.
template <typename T, typename W> hipError_t forward(const NormArgs& a, hipStream_t st) {
  auto go = [&](auto kernel, int tpr) {
    const int threads = tpr < kBlock ? kBlock : tpr, rows = threads / tpr;
    // 16 waves a CU, which the kernels' registers allow
    const int64_t blocks = (a.rows + rows - 1) / rows, most = 256 * 1024 / threads;
    return launch_kernel(kernel, dim3((unsigned)(blocks < most ? blocks : most)), threads, st, a);
  };
  constexpr int V = 16 / sizeof(T);
  if (a.cols < V) return go(norm_forward<T, W, 16, 1, 1, false>, 16);
#define RINGAR_NORM(tpr, e) \
  if (a.cols <= tpr * e) return a.stream ? go(norm_forward<T, W, tpr, e, V, true>, tpr) : go(norm_forward<T, W, tpr, e, V, false>, tpr)
  RINGAR_NORM(16, 8);
  RINGAR_NORM(64, 8);
  RINGAR_NORM(64, 16);
  RINGAR_NORM(256, 8);
  RINGAR_NORM(256, 16);
  RINGAR_NORM(512, 16);
  RINGAR_NORM(1024, 16);
#undef RINGAR_NORM
  static_assert(kNormLongest == 1024 * 16, "the widest rows held in registers");
  return launch_kernel(norm_forward_long<T, W>, dim3(capped(a.rows, 1024)), 1024, st, a);
}

template <typename T, typename W> hipError_t backward(const NormArgs& a, hipStream_t st) {
  auto go = [&](auto kernel, int threads) { return launch_kernel(kernel, dim3(a.groups), threads, st, a); };
  constexpr int V = 16 / sizeof(T);
  if (a.cols < V) return go(norm_backward<T, W, 16, 1, 1, 16, false>, 256);
#define RINGAR_NORM(tpr, e, rows)                                                                     \
  if (a.cols <= tpr * e)                                                                              \
    return a.stream ? go(norm_backward<T, W, tpr, e, V, rows, true>, tpr * rows) : go(norm_backward<T, W, tpr, e, V, rows, false>, tpr * rows)
  RINGAR_NORM(16, 8, 16);
  RINGAR_NORM(64, 8, 8);
  RINGAR_NORM(64, 16, 8);
  RINGAR_NORM(256, 8, 2);
  RINGAR_NORM(256, 16, 2);
  RINGAR_NORM(512, 16, 1);
  RINGAR_NORM(512, 32, 1);
#undef RINGAR_NORM
  hipError_t e = hipSuccess;
  if (a.y) e = launch_kernel(norm_backward_long<T, W>, dim3(capped(a.rows, 1024)), 1024, st, a);
  if (e != hipSuccess || !a.part) return e;
  return launch_kernel(norm_params_long<T>, dim3((unsigned)((a.cols + 255) / 256), a.groups), 256, st, a);
}

}  // namespace

// Blocks of the backward grid, each of which leaves one partial row: enough
// to fill the GPU (8 waves a CU), few enough that the partial rows stay small beside
// the rows themselves.  Two turns of one block cost less than a second block
// and the launch that adds their rows (16 x 832 fp16: 7.0 us, not 8.3; one
// turn 5.7).
int norm_backward_groups(int64_t rows, int cols) {
  if (cols > kNormLongest) return (int)(rows < 64 ? rows : 64);
  const int per = cols <= 128 ? 16 : cols <= 1024 ? 8 : cols <= 4096 ? 2 : 1;   // rows of a block at a time
  const int64_t blocks = (rows + per - 1) / per;
  if (blocks == 2) return 1;
  const int64_t most = cols <= 128 ? 512 : 256;
  return (int)(blocks < most ? blocks : most);
}

// Outputs that the XCDs' L2s (32 MB together) cannot hold anyway go past them
// (16384 x 8192 bf16 forward: 87 us, not 115; 16384 x 4096 backward: 70, not
// 82); smaller ones stay for whoever reads them next.
static bool beyond_l2(int dtype, const NormArgs& a) { return a.rows * a.cols * (dtype == kF32 ? 4 : 2) > 32ll << 20; }

hipError_t launch_norm_forward(int dtype, int wdtype, const NormArgs& given, hipStream_t st) {
  NormArgs a = given;
  a.stream = beyond_l2(dtype, a);
  if (dtype == kF32) return forward<float, float>(a, st);
  if (dtype == kF16) return wdtype == kF32 ? forward<_Float16, float>(a, st) : forward<_Float16, _Float16>(a, st);
  return wdtype == kF32 ? forward<__bf16, float>(a, st) : forward<__bf16, __bf16>(a, st);
}

hipError_t launch_norm_backward(int dtype, int wdtype, const NormArgs& given, hipStream_t st) {
  NormArgs a = given;
  a.stream = beyond_l2(dtype, a);
  if (dtype == kF32) return backward<float, float>(a, st);
  if (dtype == kF16) return wdtype == kF32 ? backward<_Float16, float>(a, st) : backward<_Float16, _Float16>(a, st);
  return wdtype == kF32 ? backward<__bf16, float>(a, st) : backward<__bf16, __bf16>(a, st);
}

hipError_t launch_col_sum(int out_dtype, const ColSumArgs& a, hipStream_t st) {
  const dim3 grid(capped((a.width + 63) / 64, 1024));
  if (out_dtype == kF32) return launch_kernel(col_sum<float>, grid, 1024, st, a);
  if (out_dtype == kF16) return launch_kernel(col_sum<_Float16>, grid, 1024, st, a);
  return launch_kernel(col_sum<__bf16>, grid, 1024, st, a);
}

}  // namespace ringar
