// The products' kernels for float.
#include "gemm_kernel.h"

namespace ringar {
hipError_t launch_gemm_f32(int epi, const GemmArgs& a, hipStream_t st) {
  switch (epi) {
    case kEpiLinear: return launch_general<float, kEpiLinear>(a, st);
    case kEpiGated: return launch_general<float, kEpiGated>(a, st);
    default: return launch_general<float, kEpiStore>(a, st);
  }
}
}  // namespace ringar
