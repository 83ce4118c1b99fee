// What the products' kernels share: the epilogue of one element, the matrix
// instructions of each type, and the pass that joins a product whose k was
// split.
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

// Adds the parts of a split k in order and finishes the elements.
template <typename T, int EPI> __global__ __launch_bounds__(256) void gemm_join(GemmArgs a) {
  const int64_t cols = EPI == kEpiGated ? 2 * (int64_t)a.n : a.n;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / a.n;
  const int n = (int)(i % a.n);
  if (m >= a.m) return;
  const float* p = a.part + m * cols + n;
  auto sum = [&](const float* p) { return sum_parts<4>(0, 1, a.splits, [&](int k) { return p[k * (a.m * cols)]; }); };
  const float s = sum(p);
  if constexpr (EPI == kEpiGated) finish_gated<T>(a, m, n, s, sum(p + a.n));
  else if constexpr (EPI == kEpiLinear) finish_linear<T>(a, m, n, s);
  else ((T*)a.c)[m * a.ldc + n] = (T)s;
}

}  // namespace ringar
