// Launches of one element type's products: one translation unit per type and
// operand layout.
#pragma once

#include "gemm_rows.h"
#include "gemm_tile.h"

namespace ringar {

inline unsigned blocks_of(const GemmArgs& a, int cols_of_tile, int rows_of_tile, int64_t cols) {
  return (unsigned)((cols + cols_of_tile - 1) / cols_of_tile * (((int64_t)a.m + rows_of_tile - 1) / rows_of_tile) * a.splits);
}

template <typename T, bool AROW, bool BROW, int EPI> hipError_t launch_tiled(const GemmArgs& a, hipStream_t st) {
  const int64_t cols = EPI == kEpiGated ? 2 * (int64_t)a.n : a.n;
  auto go = [&](auto kernel, int bm, int bn, int threads) {
    hipLaunchKernelGGL(kernel, dim3(blocks_of(a, bn, bm, cols)), dim3(threads), 0, st, a);
    return hipGetLastError();
  };
  switch (a.variant) {
    case kTile256:
      if constexpr (sizeof(T) == 2) return go(gemm_tile<T, AROW, BROW, EPI, 256, 256, 2, 4, 2, true>, 256, 256, 512);
      return hipErrorInvalidValue;
    case kRows:
      if constexpr (EPI != kEpiStore) {
        hipLaunchKernelGGL((gemm_rows<T, EPI, 8>), dim3((unsigned)(rows_tiles(EPI, a.n) * a.splits)), dim3(512), 0, st, a);
        return hipGetLastError();
      }
      return hipErrorInvalidValue;
    case kTile128: return go(gemm_tile<T, AROW, BROW, EPI, 128, 128, 4, 2, 4, true>, 128, 128, 512);
    case kTile64:
      if constexpr (EPI == kEpiGated) return go(gemm_tile<T, AROW, BROW, EPI, 64, 128, 2, 2, 2, true, 3>, 64, 128, 256);
      else return go(gemm_tile<T, AROW, BROW, EPI, 64, 64, 2, 2, 2, true, 3>, 64, 64, 256);
    default:
      if constexpr (EPI == kEpiGated) return go(gemm_tile<T, AROW, BROW, EPI, 64, 128, 2, 2, 2, false>, 64, 128, 256);
      else return go(gemm_tile<T, AROW, BROW, EPI, 64, 64, 2, 2, 2, false>, 64, 64, 256);
  }
}

template <typename T, int EPI> hipError_t join(const GemmArgs& a, hipStream_t st) {
  if (a.splits == 1 || a.variant == kRows) return hipSuccess;
  hipLaunchKernelGGL((gemm_join<T, EPI>), dim3((unsigned)(((int64_t)a.m * a.n + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace ringar
