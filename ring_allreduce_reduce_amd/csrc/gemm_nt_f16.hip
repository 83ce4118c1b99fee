// The forward products of Float16: x and weight both with k contiguous.
#include "gemm_launch.h"

namespace ringar {

hipError_t launch_nn_f16(const GemmArgs& a, hipStream_t st);
hipError_t launch_tn_f16(const GemmArgs& a, hipStream_t st);

template <int EPI> static hipError_t forward(const GemmArgs& a, hipStream_t st) {
  const hipError_t e = launch_tiled<_Float16, true, true, EPI>(a, st);
  return e == hipSuccess ? join<_Float16, EPI>(a, st) : e;
}

hipError_t launch_gemm_f16(int epi, const GemmArgs& a, hipStream_t st) {
  if (epi == kEpiLinear) return forward<kEpiLinear>(a, st);
  if (epi == kEpiGated) return forward<kEpiGated>(a, st);
  const hipError_t e = a.sak == 1 ? launch_nn_f16(a, st) : launch_tn_f16(a, st);
  return e == hipSuccess ? join<_Float16, kEpiStore>(a, st) : e;
}

}  // namespace ringar
