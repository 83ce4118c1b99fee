// The products' kernels for bf16.
#include "gemm_kernel.h"

namespace ringar {
hipError_t launch_gemm_bf16(int epi, const GemmArgs& a, hipStream_t st) {
  switch (epi) {
    case kEpiLinear: return launch_general<__bf16, kEpiLinear>(a, st);
    case kEpiGated: return launch_general<__bf16, kEpiGated>(a, st);
    default: return launch_general<__bf16, kEpiStore>(a, st);
  }
}
}  // namespace ringar
