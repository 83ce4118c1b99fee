// dweight = dz^T x: both operands with k as the row index (Float16).
#include "gemm_launch.h"

namespace ringar {
hipError_t launch_tn_f16(const GemmArgs& a, hipStream_t st) { return launch_tiled<_Float16, false, false, kEpiStore>(a, st); }
}  // namespace ringar
