// Launches of one element type's products: one translation unit per type and
// operand layout.
#pragma once

#include "gemm_rows.h"
#include "gemm_tile.h"

namespace ringar {

inline unsigned blocks_of(const GemmArgs& a) { return (unsigned)a.tile_count * (a.quarters ? 4 : 1) * (unsigned)a.splits; }

// A product's tiles in as many launches as their blocks need.
template <typename F> hipError_t in_parts(const GemmArgs& all, int threads, F launch_part) {
  GemmArgs a = all;
  const int64_t most = most_blocks(threads) / a.splits, end = (int64_t)a.tile_first + a.tile_count;
  hipError_t e = hipSuccess;
  for (int64_t at = a.tile_first; at < end && e == hipSuccess; at += most) {
    a.tile_first = (int)at;
    a.tile_count = (int)(end - at < most ? end - at : most);
    e = launch_part(a);
  }
  return e;
}

template <typename T, bool AROW, bool BROW, int EPI> struct Kernels {
  using Large = GemmTile<T, AROW, BROW, EPI, 256, 256, 2, 4, true>;
  using Middle = GemmTile<T, AROW, BROW, EPI, 128, 128, 4, 2, true>;
  static constexpr int kCols = EPI == kEpiGated ? 128 : 64;
  using Small = GemmTile<T, AROW, BROW, EPI, 64, kCols, 2, 2, true, 3>;
  using Staged = GemmTile<T, AROW, BROW, EPI, 64, kCols, 2, 2, false>;
};

template <typename T, bool AROW, bool BROW, int EPI> hipError_t launch_tiled(const GemmArgs& a, hipStream_t st) {
  using K = Kernels<T, AROW, BROW, EPI>;
  auto go = [&](auto kernel, int threads) {
    return in_parts(a, threads, [&](const GemmArgs& part) { return launch_kernel(kernel, dim3(blocks_of(part)), threads, st, part); });
  };
  switch (a.variant) {
    case kTile256:
      if constexpr (sizeof(T) == 2) {
        if (a.tail_count == 0) return go(gemm_tile<typename K::Large, 2>, 512);
        GemmArgs tail = a;
        tail.tile_first = a.tile_count;
        tail.tile_count = a.tail_count;
        tail.quarters = true;
        return launch_kernel(gemm_pair<typename K::Large, typename K::Middle, 2>, dim3(blocks_of(a) + blocks_of(tail)), 512, st, a, tail,
                             blocks_of(a));
      }
      return hipErrorInvalidValue;
    case kRows:
      if constexpr (EPI != kEpiStore) {
        const bool halves = ((uintptr_t)a.a | (uintptr_t)a.b | (uintptr_t)(a.sam | a.sbn) * sizeof(T)) % 4 != 0;
        if constexpr (sizeof(T) == 2) {
          if (halves) return go(gemm_rows<T, EPI, 8, true>, 512);
        }
        return go(gemm_rows<T, EPI, 8, false>, 512);
      }
      return hipErrorInvalidValue;
    case kTile128: return go(gemm_tile<typename K::Middle, 4>, 512);
    case kTile64: return go(gemm_tile<typename K::Small, 2>, 256);
    default: return go(gemm_tile<typename K::Staged, 2>, 256);
  }
}

// dx and dweight together: both of kTile128 or both of kTile64.
template <typename T> hipError_t launch_gradients(const GemmArgs& x, const GemmArgs& w, const ColSumArgs& sums, hipStream_t st) {
  const unsigned bs = (unsigned)((sums.width + 63) / 64);
  using X = Kernels<T, true, false, kEpiStore>;
  using W = Kernels<T, false, false, kEpiStore>;
  const unsigned bx = blocks_of(x), bw = blocks_of(w);
  if (x.variant == kTile128)
    return launch_kernel(gemm_gradients<T, typename X::Middle, typename W::Middle, 4>, dim3(bx + bw + bs), 512, st, x, w, sums, bx, bw);
  return launch_kernel(gemm_gradients<T, typename X::Small, typename W::Small, 2>, dim3(bx + bw + bs), 256, st, x, w, sums, bx, bw);
}

template <typename T, int EPI> hipError_t join(const GemmArgs& a, hipStream_t st) {
  if (a.splits == 1 || a.variant == kRows) return hipSuccess;
  return launch_kernel(gemm_join<T, EPI>, dim3((unsigned)(((int64_t)a.m * a.n + 255) / 256)), 256, st, a);
}

}  // namespace ringar
