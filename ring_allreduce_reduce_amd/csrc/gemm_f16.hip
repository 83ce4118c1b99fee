// The products' kernels for _Float16.
#include "gemm_kernel.h"

namespace ringar {
hipError_t launch_gemm_f16(int epi, const GemmArgs& a, hipStream_t st) {
  switch (epi) {
    case kEpiLinear: return launch_general<_Float16, kEpiLinear>(a, st);
    case kEpiGated: return launch_general<_Float16, kEpiGated>(a, st);
    default: return launch_general<_Float16, kEpiStore>(a, st);
  }
}
}  // namespace ringar
