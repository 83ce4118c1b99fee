// Both gradient products of float in one launch.
#include "gemm_launch.h"

namespace ringar {
hipError_t launch_gradients_f32(const GemmArgs& x, const GemmArgs& w, const ColSumArgs& sums, hipStream_t st) {
  hipError_t e = launch_gradients<float>(x, w, sums, st);
  if (e == hipSuccess) e = join<float, kEpiStore>(x, st);
  return e == hipSuccess ? join<float, kEpiStore>(w, st) : e;
}
}  // namespace ringar
