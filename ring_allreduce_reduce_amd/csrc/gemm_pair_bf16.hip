// Both gradient products of bf16 in one launch.
#include "gemm_launch.h"

namespace ringar {
hipError_t launch_gradients_bf16(const GemmArgs& x, const GemmArgs& w, const ColSumArgs& sums, hipStream_t st) {
  hipError_t e = launch_gradients<__bf16>(x, w, sums, st);
  if (e == hipSuccess) e = join<__bf16, kEpiStore>(x, st);
  return e == hipSuccess ? join<__bf16, kEpiStore>(w, st) : e;
}
}  // namespace ringar
