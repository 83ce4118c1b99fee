// Rows held in the registers of the threads that share them, for the norms'
// kernels.
#pragma once

#include "block_types.h"

namespace ringar {

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

// Blocks of a kernel that loops over what it has too few of.
inline unsigned capped(int64_t blocks, int threads) { return (unsigned)(blocks < most_blocks(threads) ? blocks : most_blocks(threads)); }

// Outputs (of `cols` values a row, all of them together) that the XCDs' L2s (32
// MB together) cannot hold anyway go past them (layer norm 16384 x 8192 bf16
// forward: 87 us, not 115; 16384 x 4096 backward: 70, not 82); smaller ones
// stay for whoever reads them next.
inline bool beyond_l2(int dtype, int64_t rows, int64_t cols) { return rows * cols * (dtype == kF32 ? 4 : 2) > 32ll << 20; }

}  // namespace ringar
