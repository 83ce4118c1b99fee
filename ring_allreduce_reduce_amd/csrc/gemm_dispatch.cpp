// Products by element type.
#include "block_types.h"

namespace ringar {

hipError_t launch_gemm_f16(int epi, const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_bf16(int epi, const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_f32(int epi, const GemmArgs& a, hipStream_t st);

hipError_t launch_gemm(int dtype, int epi, const GemmArgs& a, hipStream_t st) {
  if (dtype == kF16) return launch_gemm_f16(epi, a, st);
  if (dtype == kBF16) return launch_gemm_bf16(epi, a, st);
  return launch_gemm_f32(epi, a, st);
}

}  // namespace ringar
