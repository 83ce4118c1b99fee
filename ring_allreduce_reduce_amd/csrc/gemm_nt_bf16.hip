// The forward products of bf16: x and weight both with k contiguous.
#include "gemm_launch.h"

namespace ringar {

hipError_t launch_nn_bf16(const GemmArgs& a, hipStream_t st);
hipError_t launch_tn_bf16(const GemmArgs& a, hipStream_t st);

template <int EPI> static hipError_t forward(const GemmArgs& a, hipStream_t st) {
  const hipError_t e = launch_tiled<__bf16, true, true, EPI>(a, st);
  return e == hipSuccess ? join<__bf16, EPI>(a, st) : e;
}

hipError_t launch_gemm_bf16(int epi, const GemmArgs& a, hipStream_t st) {
  if (epi == kEpiLinear) return forward<kEpiLinear>(a, st);
  if (epi == kEpiGated) return forward<kEpiGated>(a, st);
  const hipError_t e = a.sak == 1 ? launch_nn_bf16(a, st) : launch_tn_bf16(a, st);
  return e == hipSuccess ? join<__bf16, kEpiStore>(a, st) : e;
}

}  // namespace ringar
