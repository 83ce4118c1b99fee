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
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) v += smem[i];
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
    u = v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) {
      u += smem[2 * i];
      v += smem[2 * i + 1];
    }
    __syncthreads();
  }
}

// E elements of a row as floats: thread t of TPR holds the packs of V
// elements that start at (i * TPR + t) * V.  Elements past the row read 0.
template <typename T, int TPR, int E>
struct Row {
  static constexpr int V = 16 / sizeof(T) < E ? 16 / sizeof(T) : E;
  static constexpr int P = E / V;
  static __device__ inline int col(int i, int t) { return (i * TPR + t) * V; }
  static __device__ inline void load(const T* p, int cols, int t, float* out, float fill = 0.0f) {
#pragma unroll
    for (int i = 0; i < P; i++) {
      const int c = col(i, t);
      if (c + V <= cols) {
        const Pack<T, V> q = load_pack<T, V>(p + c);
#pragma unroll
        for (int j = 0; j < V; j++) out[i * V + j] = (float)q.v[j];
      } else {
#pragma unroll
        for (int j = 0; j < V; j++) out[i * V + j] = c + j < cols ? (float)p[c + j] : fill;
      }
    }
  }
  // a row of another element type at the same columns
  template <typename W> static __device__ inline void load_as(const W* p, int cols, int t, float* out, float fill) {
#pragma unroll
    for (int i = 0; i < P; i++) {
      const int c = col(i, t);
      if (p != nullptr && c + V <= cols) {
        const Pack<W, V> q = load_pack<W, V>(p + c);
#pragma unroll
        for (int j = 0; j < V; j++) out[i * V + j] = (float)q.v[j];
      } else {
#pragma unroll
        for (int j = 0; j < V; j++) out[i * V + j] = p != nullptr && c + j < cols ? (float)p[c + j] : fill;
      }
    }
  }
  static __device__ inline void store(T* p, int cols, int t, const float* in) {
#pragma unroll
    for (int i = 0; i < P; i++) {
      const int c = col(i, t);
      if (c + V <= cols) {
        Pack<T, V> q;
#pragma unroll
        for (int j = 0; j < V; j++) q.v[j] = (T)in[i * V + j];
        store_pack<T, V>(p + c, q);
      } else {
#pragma unroll
        for (int j = 0; j < V; j++)
          if (c + j < cols) p[c + j] = (T)in[i * V + j];
      }
    }
  }
};

template <typename T, typename W, int TPR, int E>
__global__ __launch_bounds__(TPR < kBlock ? kBlock : TPR) void norm_forward(NormArgs a) {
  using R = Row<T, TPR, E>;
  constexpr int kThreads = TPR < kBlock ? kBlock : TPR;
  constexpr int kRows = kThreads / TPR;
  __shared__ float smem[kThreads / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  if (row >= a.rows) return;   // whole blocks where TPR > 64: a block then holds one row
  float v[E];
  R::load((const T*)a.x + row * a.ldx, a.cols, t, v);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < E; i++) s += v[i];
  const float mean = row_sum<TPR>(s, smem) * a.inv_cols;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < R::P; i++)
#pragma unroll
    for (int j = 0; j < R::V; j++) {
      float& e = v[i * R::V + j];
      e = R::col(i, t) + j < a.cols ? e - mean : 0.0f;
      s = fmaf(e, e, s);
    }
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, smem) * a.inv_cols + a.eps);
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  float w[E], b[E];
  R::template load_as<W>((const W*)a.weight, a.cols, t, w, 1.0f);
  R::template load_as<W>((const W*)a.bias, a.cols, t, b, 0.0f);
#pragma unroll
  for (int i = 0; i < E; i++) v[i] = fmaf(v[i] * rstd, w[i], b[i]);
  R::store((T*)a.y + row * a.ldy, a.cols, t, v);
}

// Rows too long for the registers: three passes, the later two from cache.
template <typename T, typename W> __global__ __launch_bounds__(1024) void norm_forward_long(NormArgs a) {
  __shared__ float smem[16];
  const int64_t row = blockIdx.x;
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

template <typename T, typename W, int TPR, int E>
__global__ __launch_bounds__(TPR < kBlock ? kBlock : TPR) void norm_backward(NormArgs a) {
  using R = Row<T, TPR, E>;
  constexpr int kThreads = TPR < kBlock ? kBlock : TPR;
  constexpr int kRows = kThreads / TPR;
  __shared__ float smem[kThreads / 64 * 2];
  const int t = threadIdx.x % TPR;
  const int lane_row = threadIdx.x / TPR;
  float w[E], dw[E], db[E];
  R::template load_as<W>((const W*)a.weight, a.cols, t, w, 1.0f);
#pragma unroll
  for (int i = 0; i < E; i++) dw[i] = db[i] = 0.0f;
  // every thread of a block runs the same number of turns; a row past the
  // end is computed on zeros and not stored
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += (int64_t)a.groups * kRows) {
    const int64_t row = base + lane_row;
    const bool live = row < a.rows;
    float h[E], dy[E];
    float mean = 0.0f, rstd = 0.0f;
    if (live) {
      R::load((const T*)a.x + row * a.ldx, a.cols, t, h);
      R::load((const T*)a.dy + row * a.lddy, a.cols, t, dy);
      mean = a.mean[row];
      rstd = a.rstd[row];
    } else {
#pragma unroll
      for (int i = 0; i < E; i++) h[i] = dy[i] = 0.0f;
    }
    float sg = 0.0f, sgh = 0.0f;
#pragma unroll
    for (int i = 0; i < R::P; i++)
#pragma unroll
      for (int j = 0; j < R::V; j++) {
        const int e = i * R::V + j;
        h[e] = R::col(i, t) + j < a.cols ? (h[e] - mean) * rstd : 0.0f;
        dw[e] = fmaf(dy[e], h[e], dw[e]);
        db[e] += dy[e];
        dy[e] *= w[e];
        sg += dy[e];
        sgh = fmaf(dy[e], h[e], sgh);
      }
    if (a.y) {
      row_sum2<TPR>(sg, sgh, smem);
      sg *= a.inv_cols;
      sgh *= a.inv_cols;
#pragma unroll
      for (int i = 0; i < E; i++) dy[i] = rstd * (dy[i] - sg - h[i] * sgh);
      if (live) R::store((T*)a.y + row * a.ldy, a.cols, t, dy);
    }
  }
  if (!a.part) return;
  // the block's rows into one partial row
  if constexpr (kRows > 1) {
    __shared__ float rows[kRows][TPR * E];
#pragma unroll
    for (int which = 0; which < 2; which++) {
      if (which) __syncthreads();
#pragma unroll
      for (int i = 0; i < R::P; i++)
#pragma unroll
        for (int j = 0; j < R::V; j++) rows[lane_row][R::col(i, t) + j] = which ? db[i * R::V + j] : dw[i * R::V + j];
      __syncthreads();
      float* out = a.part + ((int64_t)which * a.groups + blockIdx.x) * a.cols;
      for (int c = threadIdx.x; c < TPR * E && c < a.cols; c += kThreads) {
        float s = 0.0f;
#pragma unroll 4
        for (int r = 0; r < kRows; r++) s += rows[r][c];
        out[c] = s;
      }
    }
  } else {
    float* out = a.part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
    for (int i = 0; i < R::P; i++)
#pragma unroll
      for (int j = 0; j < R::V; j++) {
        const int c = R::col(i, t) + j;
        if (c < a.cols) {
          out[c] = dw[i * R::V + j];
          out[(int64_t)a.groups * a.cols + c] = db[i * R::V + j];
        }
      }
  }
}

// dx of rows too long for the registers
template <typename T, typename W> __global__ __launch_bounds__(1024) void norm_backward_long(NormArgs a) {
  __shared__ float smem[32];
  const int64_t row = blockIdx.x;
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
  a.part[(int64_t)blockIdx.y * a.cols + c] = dw;
  a.part[((int64_t)a.groups + blockIdx.y) * a.cols + c] = db;
}

template <typename O> __global__ __launch_bounds__(256) void col_sum(ColSumArgs a) {
  __shared__ float smem[4][64];
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  float s = 0.0f;
  if (c < a.cols)
    for (int p = w; p < a.parts; p += 4) s += a.part[p * a.cols + c];
  smem[w][threadIdx.x & 63] = s;
  __syncthreads();
  if (w == 0 && c < a.cols)
    ((O*)a.out)[c] = (O)((smem[0][threadIdx.x] + smem[1][threadIdx.x]) + (smem[2][threadIdx.x] + smem[3][threadIdx.x]));
}

// Threads and elements per thread of a row: the smallest shape that holds it.
constexpr int kLongest = 1024 * 16;
template <typename T, typename W> hipError_t forward(const NormArgs& a, hipStream_t st) {
  auto go = [&](auto kernel, int tpr) {
    const int threads = tpr < kBlock ? kBlock : tpr, rows = threads / tpr;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((a.rows + rows - 1) / rows)), dim3(threads), 0, st, a);
    return hipGetLastError();
  };
  if (a.cols <= 16 * 8) return go(norm_forward<T, W, 16, 8>, 16);
  if (a.cols <= 64 * 8) return go(norm_forward<T, W, 64, 8>, 64);
  if (a.cols <= 64 * 16) return go(norm_forward<T, W, 64, 16>, 64);
  if (a.cols <= 256 * 8) return go(norm_forward<T, W, 256, 8>, 256);
  if (a.cols <= 256 * 16) return go(norm_forward<T, W, 256, 16>, 256);
  if (a.cols <= 512 * 16) return go(norm_forward<T, W, 512, 16>, 512);
  if (a.cols <= kLongest) return go(norm_forward<T, W, 1024, 16>, 1024);
  hipLaunchKernelGGL((norm_forward_long<T, W>), dim3((unsigned)a.rows), dim3(1024), 0, st, a);
  return hipGetLastError();
}

template <typename T, typename W> hipError_t backward(const NormArgs& a, hipStream_t st) {
  auto go = [&](auto kernel, int tpr) {
    hipLaunchKernelGGL(kernel, dim3(a.groups), dim3(tpr < kBlock ? kBlock : tpr), 0, st, a);
    return hipGetLastError();
  };
  if (a.cols <= 16 * 8) return go(norm_backward<T, W, 16, 8>, 16);
  if (a.cols <= 64 * 8) return go(norm_backward<T, W, 64, 8>, 64);
  if (a.cols <= 64 * 16) return go(norm_backward<T, W, 64, 16>, 64);
  if (a.cols <= 256 * 8) return go(norm_backward<T, W, 256, 8>, 256);
  if (a.cols <= 256 * 16) return go(norm_backward<T, W, 256, 16>, 256);
  if (a.cols <= 512 * 16) return go(norm_backward<T, W, 512, 16>, 512);
  if (a.cols <= kLongest) return go(norm_backward<T, W, 1024, 16>, 1024);
  if (a.y) {
    hipLaunchKernelGGL((norm_backward_long<T, W>), dim3((unsigned)a.rows), dim3(1024), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
  }
  if (a.part) hipLaunchKernelGGL((norm_params_long<T>), dim3((unsigned)((a.cols + 255) / 256), a.groups), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

int norm_backward_groups(int dtype, int64_t rows, int cols) {
  (void)dtype;
  const int per = cols <= 128 ? 16 : cols <= 1024 ? 4 : 1;   // rows of a block at a time
  const int64_t blocks = (rows + per - 1) / per;
  const int most = cols <= kLongest ? 512 : 64;
  return (int)(blocks < most ? blocks : most);
}

hipError_t launch_norm_forward(int dtype, int wdtype, const NormArgs& a, hipStream_t st) {
  if (dtype == kF32) return forward<float, float>(a, st);
  if (dtype == kF16) return wdtype == kF32 ? forward<_Float16, float>(a, st) : forward<_Float16, _Float16>(a, st);
  return wdtype == kF32 ? forward<__bf16, float>(a, st) : forward<__bf16, __bf16>(a, st);
}

hipError_t launch_norm_backward(int dtype, int wdtype, const NormArgs& a, hipStream_t st) {
  if (dtype == kF32) return backward<float, float>(a, st);
  if (dtype == kF16) return wdtype == kF32 ? backward<_Float16, float>(a, st) : backward<_Float16, _Float16>(a, st);
  return wdtype == kF32 ? backward<__bf16, float>(a, st) : backward<__bf16, __bf16>(a, st);
}

hipError_t launch_col_sum(int out_dtype, const ColSumArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.cols + 63) / 64));
  if (out_dtype == kF32) hipLaunchKernelGGL(col_sum<float>, grid, dim3(256), 0, st, a);
  else if (out_dtype == kF16) hipLaunchKernelGGL(col_sum<_Float16>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(col_sum<__bf16>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace ringar
