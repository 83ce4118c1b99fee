// Root-mean-square norm joined to the residual stream, forward and backward.
//
//   s = x + residual (rounded to its type: what is stored and what is normed),
//   r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   8 bits: scale = max |y| / 448 over a row or 128 columns of it, q = y / scale
//   g = dy w,  h = s r,  dx = r (g - h mean(g h)) + dsum,  dw = sum dy h
//
// Rows lie in registers as in the layer norm's kernels (norm_rows.h): memory
// sees every input and output once, one sum over the row's threads a row
// (8 bits: and a maximum), fp32 throughout.  A group of 128 columns lies in 16
// (fp32: 32) neighbouring lanes of one wave, so its maximum needs no LDS.
//
// Memory bound.  A call takes, forward with a residual 16384 x 8192 bf16 197 us
// (5.5 TB/s), in 8 bits with a scale for each 128 columns 2053 x 5120 fp16 18 us
// (4.1 TB/s), backward 16384 x 4096 bf16 with its column sums 100 us (5.4 TB/s).
#include "layer_types.h"
#include "norm_rows.h"

namespace ringar {
namespace {

// Larger of magnitudes by their bits, which order like the values and put NaN
// above infinity: a NaN is not lost.
__device__ inline uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
__device__ inline uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int LANES> __device__ inline uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = larger(v, __shfl_xor(v, o));
  return v;
}

template <int TPR> __device__ inline uint32_t row_max(uint32_t v, float* smem) {
  v = lanes_max<(TPR < 64 ? TPR : 64)>(v);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    uint32_t* s = (uint32_t*)smem;
    if ((threadIdx.x & 63) == 0) s[wave] = v;
    __syncthreads();
    const uint32_t* row = s + wave / (TPR / 64) * (TPR / 64);
    v = 0;
#pragma unroll
    for (int i = 0; i < TPR / 64; i++) v = larger(v, row[i]);
    __syncthreads();
  }
  return v;
}

__device__ inline float scale_of(uint32_t most) {
  const float s = __builtin_bit_cast(float, most) / kLargest8;
  return s < kLeastScale ? kLeastScale : s;
}

// Four values as four 8-bit ones, rounded to nearest even.  Their magnitude is
// at most 448 (1 + 2^-22), which rounds to 448.
__device__ inline uint32_t four8(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}
__device__ inline uint8_t one8(float a) { return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, a, 0, false); }

template <typename R, int V, int P> __device__ inline void store8(const R& r, uint8_t* p, const float* in) {
#pragma unroll
  for (int i = 0; i < P; i++) {
    if (V % 4 == 0 && r.skip[i] == 0) {
      uint32_t w[V / 4 + (V < 4)];
#pragma unroll
      for (int j = 0; j + 4 <= V; j += 4) w[j / 4] = four8(in[i * V + j], in[i * V + j + 1], in[i * V + j + 2], in[i * V + j + 3]);
      __builtin_memcpy(p + r.col[i], w, V);
    } else {
#pragma unroll
      for (int j = 0; j < V; j++)
        if (j >= r.skip[i]) p[r.col[i] + j] = one8(in[i * V + j]);
    }
  }
}

template <typename T, typename W, int TPR, int E, int V, int OUT, bool STREAM>
__global__ __launch_bounds__(TPR < kBlock ? kBlock : TPR) void rms_forward(RmsArgs a) {
  using R = Row<T, TPR, E, V>;
  constexpr int kThreads = TPR < kBlock ? kBlock : TPR;
  constexpr int kRows = kThreads / TPR;
  __shared__ float smem[kThreads / 64];
  const int t = threadIdx.x % TPR;
  const R r(a.cols, t);
  // A block takes rows in turn, as the layer norm's does: the weight stays in
  // registers, the next row is on its way while this one is worked on, and a
  // row past the end is the last one again and not stored.
  const int64_t stride = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  typename R::template Raw<T> next, more;
  typename R::template Raw<W> w;
  auto fetch = [&](int64_t i) {
    i = i < a.rows ? i : a.rows - 1;
    r.template load<T>((const T*)a.x + i * a.ldx, next);
    if (a.residual) r.template load<T>((const T*)a.residual + i * a.ldr, more);
  };
  fetch(row);
  if (a.weight) r.template load<W>((const W*)a.weight, w);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride, row += stride) {
    float v[E];
    r.template widen<T>(next, v);
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < E; i++) v[i] = (float)(T)(v[i] + (float)more.q[i / V].v[i % V]);
      r.clear(v);
    }
    fetch(row + stride);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i++) s = fmaf(v[i], v[i], s);
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, smem) * a.inv_cols + a.eps);
    const bool live = row < a.rows;
    if (live) {
      if (t == 0 && a.rstd) a.rstd[row] = rstd;
      if (a.residual) r.template store<STREAM>((T*)a.sum + row * a.lds, v);
    }
#pragma unroll
    for (int i = 0; i < E; i++) v[i] = v[i] * rstd * (a.weight ? (float)w.q[i / V].v[i % V] : 1.0f);
    if constexpr (OUT == kOutSame) {
      if (live) r.template store<STREAM>((T*)a.y + row * a.ldy, v);
    } else {
      r.clear(v);                    // an infinite weight makes NaN of a zero
      uint8_t* y = (uint8_t*)a.y + row * a.ldy;
      if constexpr (OUT == kOutRow8) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < E; i++) most = larger(most, magnitude(v[i]));
        const float scale = scale_of(row_max<TPR>(most, smem));
        if (t == 0 && live) a.scale[row] = scale;
        const float inv = 1.0f / scale;
#pragma unroll
        for (int i = 0; i < E; i++) v[i] *= inv;
      } else {
        constexpr int kLanes = kScaleGroup / V;
#pragma unroll
        for (int i = 0; i < E / V; i++) {
          uint32_t most = 0;
#pragma unroll
          for (int j = 0; j < V; j++) most = larger(most, magnitude(v[i * V + j]));
          const float scale = scale_of(lanes_max<kLanes>(most));
          const int c = (i * TPR + t) * V;
          if (t % kLanes == 0 && c < a.cols && live) a.scale[row * a.scales + c / kScaleGroup] = scale;
          const float inv = 1.0f / scale;
#pragma unroll
          for (int j = 0; j < V; j++) v[i * V + j] *= inv;
        }
      }
      if (live) store8<R, V, E / V>(r, y, v);
    }
  }
}

// Rows too long for the registers: a pass for the sum and its square, the
// others from cache, value by value.
template <typename T, typename W> __global__ __launch_bounds__(1024) void rms_forward_long(RmsArgs a) {
  __shared__ float smem[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    float s = 0.0f;
    // a thread reads in the later passes what it has written in this one
    const T* from = a.residual ? (const T*)a.sum + row * a.lds : x;
    auto each = [&](auto f) {
      for (int64_t c = (int64_t)wave * kScaleGroup + lane; c < a.cols; c += 16 * kScaleGroup) {
        f(c);
        if (c + 64 < a.cols) f(c + 64);
      }
    };
    each([&](int64_t c) {
      float v = (float)x[c];
      if (a.residual) {
        const T sum = (T)(v + (float)((const T*)a.residual)[row * a.ldr + c]);
        ((T*)a.sum)[row * a.lds + c] = sum;
        v = (float)sum;
      }
      s = fmaf(v, v, s);
    });
    const float rstd = 1.0f / sqrtf(row_sum<1024>(s, smem) * a.inv_cols + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    auto value = [&](int64_t c) { return (float)from[c] * rstd * (a.weight ? (float)((const W*)a.weight)[c] : 1.0f); };
    if (a.out == kOutSame) {
      each([&](int64_t c) { ((T*)a.y)[row * a.ldy + c] = (T)value(c); });
    } else if (a.out == kOutRow8) {
      uint32_t most = 0;
      each([&](int64_t c) { most = larger(most, magnitude(value(c))); });
      const float scale = scale_of(row_max<1024>(most, smem)), inv = 1.0f / scale;
      if (threadIdx.x == 0) a.scale[row] = scale;
      each([&](int64_t c) { ((uint8_t*)a.y)[row * a.ldy + c] = one8(value(c) * inv); });
    } else {
      // a wave takes a group at a time, two values a lane
      for (int64_t g = wave; g < a.scales; g += 16) {
        const int64_t c = g * kScaleGroup + lane;
        const float u = c < a.cols ? value(c) : 0.0f, v = c + 64 < a.cols ? value(c + 64) : 0.0f;
        const float scale = scale_of(lanes_max<64>(larger(magnitude(u), magnitude(v)))), inv = 1.0f / scale;
        if (lane == 0) a.scale[row * a.scales + g] = scale;
        uint8_t* y = (uint8_t*)a.y + row * a.ldy;
        if (c < a.cols) y[c] = one8(u * inv);
        if (c + 64 < a.cols) y[c + 64] = one8(v * inv);
      }
    }
  }
}

template <typename T, typename W, int TPR, int E, int V, int kRows, bool STREAM>
__global__ __launch_bounds__(TPR * kRows) void rms_backward(RmsArgs a) {
  using R = Row<T, TPR, E, V>;
  constexpr int kThreads = TPR * kRows;
  constexpr bool kAhead = E < 32;        // as in the layer norm's: longer rows leave no registers
  __shared__ float smem[kThreads / 64];
  const int t = threadIdx.x % TPR;
  const int lane_row = threadIdx.x / TPR;
  const R r(a.cols, t);
  const int64_t stride = (int64_t)a.blocks * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + lane_row;
  typename R::template Raw<T> rx, rdy, rds;
  float next_rstd;
  auto fetch = [&](int64_t i) {
    i = i < a.rows ? i : a.rows - 1;
    r.template load<T>((const T*)a.x + i * a.ldx, rx);
    r.template load<T>((const T*)a.dy + i * a.lddy, rdy);
    if (a.residual) r.template load<T>((const T*)a.residual + i * a.ldr, rds);
    next_rstd = a.rstd[i];
  };
  if (kAhead) fetch(row);
  float dw[E];
  typename R::template Raw<W> wt;
  if (a.weight) r.template load<W>((const W*)a.weight, wt);
#pragma unroll
  for (int i = 0; i < E; i++) dw[i] = 0.0f;
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride, row += stride) {
    const bool live = row < a.rows;
    if (!kAhead) fetch(row);
    float h[E], dy[E], ds[E];
    r.template widen<T>(rx, h);
    r.template widen<T>(rdy, dy);
    if (a.residual) {
      r.template widen<T>(rds, ds);
    } else {
#pragma unroll
      for (int i = 0; i < E; i++) ds[i] = 0.0f;
    }
    const float rstd = next_rstd;
    if (kAhead) fetch(row + stride);
    float sgh = 0.0f;
#pragma unroll
    for (int i = 0; i < E; i++) {
      dy[i] = live ? dy[i] : 0.0f;
      h[i] = live ? h[i] * rstd : 0.0f;
      dw[i] = fmaf(dy[i], h[i], dw[i]);      // both are 0 where a pack holds no element
      dy[i] *= a.weight ? (float)wt.q[i / V].v[i % V] : 1.0f;
      sgh = fmaf(dy[i], h[i], sgh);
    }
    if (a.y) {
      sgh = row_sum<TPR>(sgh, smem) * a.inv_cols;
#pragma unroll
      for (int i = 0; i < E; i++) dy[i] = fmaf(rstd, dy[i] - h[i] * sgh, ds[i]);
      if (live) r.template store<STREAM>((T*)a.y + row * a.ldy, dy);
    }
  }
  if (!a.part && !a.dweight) return;
  // the block's rows into one partial row, or where it has them all into the gradient
  float* out = a.part + (int64_t)blockIdx.x * a.cols;
  auto put = [&](int c, float s) {
    if (a.part) out[c] = s;
    else ((W*)a.dweight)[c] = (W)s;
  };
  if constexpr (kRows > 1) {
    __shared__ float rows[kRows][TPR * E];
    r.sums(rows[lane_row], dw);
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kThreads) {
      float s = 0.0f;
#pragma unroll 4
      for (int i = 0; i < kRows; i++) s += rows[i][c];
      put(c, s);
    }
  } else {
    if (a.part) r.sums(out, dw);
    else r.each([&](int i, int c) { put(c, dw[i]); });
  }
}

// dx of rows too long for the registers
template <typename T, typename W> __global__ __launch_bounds__(1024) void rms_backward_long(RmsArgs a) {
  __shared__ float smem[16];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* dy = (const T*)a.dy + row * a.lddy;
    const float rstd = a.rstd[row];
    auto g = [&](int64_t c) { return (float)dy[c] * (a.weight ? (float)((const W*)a.weight)[c] : 1.0f); };
    float sgh = 0.0f;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) sgh = fmaf(g(c), (float)x[c] * rstd, sgh);
    sgh = row_sum<1024>(sgh, smem) * a.inv_cols;
    T* dx = (T*)a.y + row * a.ldy;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
      const float ds = a.residual ? (float)((const T*)a.residual)[row * a.ldr + c] : 0.0f;
      dx[c] = (T)fmaf(rstd, g(c) - (float)x[c] * rstd * sgh, ds);
    }
  }
}

// the weight's gradient of such rows: one column a thread, the block's rows in turn
template <typename T> __global__ __launch_bounds__(256) void rms_params_long(RmsArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += a.blocks)
    dw = fmaf((float)((const T*)a.dy)[row * a.lddy + c], (float)((const T*)a.x)[row * a.ldx + c] * a.rstd[row], dw);
  a.part[(int64_t)blockIdx.y * a.cols + c] = dw;
}

template <typename T, typename W, int OUT> hipError_t forward_as(const RmsArgs& a, hipStream_t st) {
  auto go = [&](auto kernel, int tpr) {
    const int threads = tpr < kBlock ? kBlock : tpr, rows = threads / tpr;
    const int64_t blocks = (a.rows + rows - 1) / rows, most = 256 * 1024 / threads;
    return launch_kernel(kernel, dim3((unsigned)(blocks < most ? blocks : most)), threads, st, a);
  };
  constexpr int V = 16 / sizeof(T);
  if constexpr (OUT != kOutGroup8) {
    if (a.cols < V) return go(rms_forward<T, W, 16, 1, 1, OUT, false>, 16);
#define RINGAR_RMS(tpr, e) \
  if (a.cols <= tpr * e) return a.stream ? go(rms_forward<T, W, tpr, e, V, OUT, true>, tpr) : go(rms_forward<T, W, tpr, e, V, OUT, false>, tpr)
    RINGAR_RMS(16, 8);
  }
  // (groups: more than 128 columns)
  RINGAR_RMS(64, 8);
  RINGAR_RMS(64, 16);
  RINGAR_RMS(256, 8);
  RINGAR_RMS(256, 16);
  RINGAR_RMS(512, 16);
  RINGAR_RMS(1024, 16);
#undef RINGAR_RMS
  static_assert(kNormLongest == 1024 * 16, "the widest rows held in registers");
  return launch_kernel(rms_forward_long<T, W>, dim3(capped(a.rows, 1024)), 1024, st, a);
}

template <typename T, typename W> hipError_t forward(const RmsArgs& a, hipStream_t st) {
  if (a.out == kOutSame) return forward_as<T, W, kOutSame>(a, st);
  if (a.out == kOutRow8) return forward_as<T, W, kOutRow8>(a, st);
  return forward_as<T, W, kOutGroup8>(a, st);
}

template <typename T, typename W> hipError_t backward(const RmsArgs& a, hipStream_t st) {
  auto go = [&](auto kernel, int threads) { return launch_kernel(kernel, dim3(a.blocks), threads, st, a); };
  constexpr int V = 16 / sizeof(T);
  if (a.cols < V) return go(rms_backward<T, W, 16, 1, 1, 16, false>, 256);
#define RINGAR_RMS(tpr, e, rows)                                                                     \
  if (a.cols <= tpr * e)                                                                             \
    return a.stream ? go(rms_backward<T, W, tpr, e, V, rows, true>, tpr * rows) : go(rms_backward<T, W, tpr, e, V, rows, false>, tpr * rows)
  RINGAR_RMS(16, 8, 16);
  RINGAR_RMS(64, 8, 8);
  RINGAR_RMS(64, 16, 8);
  RINGAR_RMS(256, 8, 2);
  RINGAR_RMS(256, 16, 2);
  RINGAR_RMS(512, 16, 1);
  RINGAR_RMS(512, 32, 1);
#undef RINGAR_RMS
  hipError_t e = hipSuccess;
  if (a.y) e = launch_kernel(rms_backward_long<T, W>, dim3(capped(a.rows, 1024)), 1024, st, a);
  if (e != hipSuccess || !a.part) return e;
  return launch_kernel(rms_params_long<T>, dim3((unsigned)((a.cols + 255) / 256), a.blocks), 256, st, a);
}

}  // namespace

// Blocks of the backward grid: the layer norm's count.
int rms_backward_blocks(int64_t rows, int cols) { return norm_backward_groups(rows, cols); }

// (The sum and y together: 4096 x 4096 bf16 with a residual 25 us past the
// caches, not 28.)
hipError_t launch_rms_forward(int dtype, int wdtype, const RmsArgs& given, hipStream_t st) {
  RmsArgs a = given;
  const int64_t size = dtype == kF32 ? 4 : 2, sum = a.residual ? a.cols : 0, y = a.out == kOutSame ? a.cols : a.cols / size;
  a.stream = beyond_l2(dtype, a.rows, sum + y);
  if (dtype == kF32) return forward<float, float>(a, st);
  if (dtype == kF16) return wdtype == kF32 ? forward<_Float16, float>(a, st) : forward<_Float16, _Float16>(a, st);
  return wdtype == kF32 ? forward<__bf16, float>(a, st) : forward<__bf16, __bf16>(a, st);
}

hipError_t launch_rms_backward(int dtype, int wdtype, const RmsArgs& given, hipStream_t st) {
  RmsArgs a = given;
  a.stream = beyond_l2(dtype, a.rows, a.cols);
  if (dtype == kF32) return backward<float, float>(a, st);
  if (dtype == kF16) return wdtype == kF32 ? backward<_Float16, float>(a, st) : backward<_Float16, _Float16>(a, st);
  return wdtype == kF32 ? backward<__bf16, float>(a, st) : backward<__bf16, __bf16>(a, st);
}

}  // namespace ringar
