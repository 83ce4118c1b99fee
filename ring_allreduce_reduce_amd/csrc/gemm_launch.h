// Launches of one element type's products: one translation unit per type and
// operand layout.
#pragma once

#include "gemm_tile.h"

namespace ringar {

inline unsigned blocks_of(const GemmArgs& a, int cols_of_tile, int rows_of_tile, int64_t cols) {
  return (unsigned)((cols + cols_of_tile - 1) / cols_of_tile * (((int64_t)a.m + rows_of_tile - 1) / rows_of_tile) * a.splits);
}

template <typename T, int EPI> hipError_t launch_general(const GemmArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((gemm_general<T, EPI>), dim3(blocks_of(a, 64, 64, logical_cols(EPI, a.n))), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <typename T, bool AROW, bool BROW, int EPI> hipError_t launch_tiled(const GemmArgs& a, hipStream_t st) {
  const int64_t cols = EPI == kEpiGated ? 2 * (int64_t)a.n : a.n;
  if (a.variant == kTile256) {
    if constexpr (sizeof(T) == 2)
      hipLaunchKernelGGL((gemm_tile<T, AROW, BROW, EPI, 256, 256, 2, 4, 2>), dim3(blocks_of(a, 256, 256, cols)), dim3(512), 0, st, a);
  } else if (a.variant == kTile128) {
    hipLaunchKernelGGL((gemm_tile<T, AROW, BROW, EPI, 128, 128, 2, 2, 2>), dim3(blocks_of(a, 128, 128, cols)), dim3(256), 0, st, a);
  } else {
    if constexpr (AROW)
      hipLaunchKernelGGL((gemm_tile<T, AROW, BROW, EPI, 64, 128, 1, 2, 1>), dim3(blocks_of(a, 128, 64, cols)), dim3(128), 0, st, a);
  }
  return hipGetLastError();
}

template <typename T, int EPI> hipError_t join(const GemmArgs& a, hipStream_t st) {
  if (a.splits == 1) return hipSuccess;
  hipLaunchKernelGGL((gemm_join<T, EPI>), dim3((unsigned)(((int64_t)a.m * a.n + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace ringar
