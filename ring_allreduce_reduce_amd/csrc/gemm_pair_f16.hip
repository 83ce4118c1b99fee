// Both gradient products of Float16 in one launch.
#include "gemm_launch.h"

namespace ringar {
hipError_t launch_gradients_f16(const GemmArgs& x, const GemmArgs& w, const ColSumArgs& sums, hipStream_t st) {
  hipError_t e = launch_gradients<_Float16>(x, w, sums, st);
  if (e == hipSuccess) e = join<_Float16, kEpiStore>(x, st);
  return e == hipSuccess ? join<_Float16, kEpiStore>(w, st) : e;
}
}  // namespace ringar
