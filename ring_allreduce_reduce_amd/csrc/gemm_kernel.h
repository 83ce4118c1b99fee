// Products with fused epilogues: the kernel that takes any strides, the pass
// that joins a product whose k was split, and the epilogues they share.
#pragma once

#include "block_types.h"

namespace ringar {

// ---------------------------------------------------------------- epilogue
// One output element: bias, activation, residual (fp32, one rounding at the
// end; the pre-activation is rounded once for the backward pass).
template <typename T> __device__ inline void finish_linear(const GemmArgs& a, int64_t m, int n, float z) {
  constexpr bool kFast = sizeof(T) == 2;
  if (a.bias) z += (float)((const T*)a.bias)[n];
  if (a.pre) ((T*)a.pre)[m * a.ldp + n] = (T)z;
  z = activate<kFast>(a.act, z);
  if (a.residual) z += (float)((const T*)a.residual)[m * a.ldr + n];
  ((T*)a.c)[m * a.ldc + n] = (T)z;
}

template <typename T> __device__ inline void finish_gated(const GemmArgs& a, int64_t m, int n, float g, float u) {
  constexpr bool kFast = sizeof(T) == 2;
  if (a.bias) {
    g += (float)((const T*)a.bias)[n];
    u += (float)((const T*)a.bias)[a.n + n];
  }
  if (a.pre) {
    ((T*)a.pre)[m * a.ldp + n] = (T)g;
    ((T*)a.pre)[m * a.ldp + a.n + n] = (T)u;
  }
  ((T*)a.c)[m * a.ldc + n] = (T)(activate<kFast>(a.act, g) * u);
}

// row of B that logical column l stands for; -1: none
template <int EPI> __device__ inline int64_t b_row(const GemmArgs& a, int64_t l) {
  if constexpr (EPI == kEpiGated) {
    const int64_t c = (l >> 5) * 16 + (l & 15);
    return c < a.n ? (l & 16 ? a.n + c : c) : -1;
  }
  return l < a.n ? l : -1;
}

// ------------------------------------------------------- matrix instructions
// One 16 x 16 block of C gains the products over KSTEP values of k.  Lane l
// holds KSTEP / 4 values of row (column) l % 16; which ones is the same on
// both sides, so their order does not matter.  The result's lane l holds
// rows l / 16 * 4 .. + 3 of the first operand, column l % 16 of the second.
template <typename T> struct Mma;
template <> struct Mma<_Float16> {
  typedef _Float16 Frag __attribute__((ext_vector_type(8)));
  static __device__ inline f32x4 run(Frag a, Frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};
template <> struct Mma<__bf16> {
  typedef __bf16 Frag __attribute__((ext_vector_type(8)));
  static __device__ inline f32x4 run(Frag a, Frag b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Mma<float> {
  typedef float Frag __attribute__((ext_vector_type(4)));
  static __device__ inline f32x4 run(Frag a, Frag b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; i++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

// ------------------------------------------------------------ general kernel
// 64 x 64 tile of C, four waves of 32 x 32.  Operands come element by
// element through registers into LDS (zeros past every edge), so any strides
// and alignment will do.
template <typename T, int EPI> __global__ __launch_bounds__(256) void gemm_general(GemmArgs a) {
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kStep = 4 * kVec;             // k of one fragment
  constexpr int kPitch = kStep + kVec;        // rows shifted over the banks
  __shared__ __attribute__((aligned(16))) T sa[64 * kPitch];
  __shared__ __attribute__((aligned(16))) T sb[64 * kPitch];
  using Frag = typename Mma<T>::Frag;
  const int64_t cols = logical_cols(EPI, a.n);
  const int64_t tiles_n = (cols + 63) / 64;
  const int64_t tiles = tiles_n * ((a.m + 63) / 64);
  const int64_t tile = blockIdx.x % tiles;
  const int split = (int)(blockIdx.x / tiles);
  const int64_t m0 = tile / tiles_n * 64, n0 = tile % tiles_n * 64;
  const int k_begin = split * a.k_per_split;
  const int k_end = a.k - k_begin < a.k_per_split ? a.k : k_begin + a.k_per_split;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
  const int64_t part_cols = EPI == kEpiGated ? 2 * (int64_t)a.n : a.n;
  f32x4 acc[2][2] = {};
  for (int k0 = k_begin; k0 < k_end; k0 += kStep) {
    __syncthreads();
    // the index with stride 1 runs along the threads
#pragma unroll
    for (int i = 0; i < 64 * kStep / 256; i++) {
      const int e = i * 256 + threadIdx.x;
      {
        const int r = a.sak == 1 ? e / kStep : e % 64, k = a.sak == 1 ? e % kStep : e / 64;
        const int64_t m = m0 + r;
        sa[r * kPitch + k] = m < a.m && k0 + k < k_end ? ((const T*)a.a)[m * a.sam + (k0 + k) * a.sak] : (T)0.0f;
      }
      {
        const int r = a.sbk == 1 ? e / kStep : e % 64, k = a.sbk == 1 ? e % kStep : e / 64;
        const int64_t n = b_row<EPI>(a, n0 + r);
        sb[r * kPitch + k] = n >= 0 && k0 + k < k_end ? ((const T*)a.b)[n * a.sbn + (k0 + k) * a.sbk] : (T)0.0f;
      }
    }
    __syncthreads();
    Frag fa[2], fb[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      fa[i] = *(const Frag*)(sa + (wm + i * 16 + (lane & 15)) * kPitch + (lane >> 4) * kVec);
      fb[i] = *(const Frag*)(sb + (wn + i * 16 + (lane & 15)) * kPitch + (lane >> 4) * kVec);
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int j = 0; j < 2; j++) acc[i][j] = Mma<T>::run(fa[i], fb[j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int64_t m = m0 + wm + i * 16 + (lane >> 4) * 4 + r;
      if (m >= a.m) continue;
      if (a.splits > 1) {
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const int64_t n = b_row<EPI>(a, n0 + wn + j * 16 + (lane & 15));
          if (n >= 0) a.part[((int64_t)split * a.m + m) * part_cols + n] = acc[i][j][r];
        }
      } else if constexpr (EPI == kEpiGated) {
        const int64_t n = (n0 + wn) / 2 + (lane & 15);
        if (n < a.n) finish_gated<T>(a, m, (int)n, acc[i][0][r], acc[i][1][r]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const int64_t n = n0 + wn + j * 16 + (lane & 15);
          if (n >= a.n) continue;
          if constexpr (EPI == kEpiLinear) finish_linear<T>(a, m, (int)n, acc[i][j][r]);
          else ((T*)a.c)[m * a.ldc + n] = (T)acc[i][j][r];
        }
      }
    }
}

// Adds the parts of a split k in order and finishes the elements.
template <typename T, int EPI> __global__ __launch_bounds__(256) void gemm_join(GemmArgs a) {
  const int64_t cols = EPI == kEpiGated ? 2 * (int64_t)a.n : a.n;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / a.n;
  const int n = (int)(i % a.n);
  if (m >= a.m) return;
  const float* p = a.part + m * cols + n;
  float s = 0.0f, u = 0.0f;
  for (int k = 0; k < a.splits; k++) {
    s += p[(int64_t)k * a.m * cols];
    if constexpr (EPI == kEpiGated) u += p[(int64_t)k * a.m * cols + a.n];
  }
  if constexpr (EPI == kEpiGated) finish_gated<T>(a, m, n, s, u);
  else if constexpr (EPI == kEpiLinear) finish_linear<T>(a, m, n, s);
  else ((T*)a.c)[m * a.ldc + n] = (T)s;
}

}  // namespace ringar
