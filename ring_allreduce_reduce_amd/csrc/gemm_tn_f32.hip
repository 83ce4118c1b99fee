// dweight = dz^T x: both operands with k as the row index (float).
#include "gemm_launch.h"

namespace ringar {
hipError_t launch_tn_f32(const GemmArgs& a, hipStream_t st) { return launch_tiled<float, false, false, kEpiStore>(a, st); }
}  // namespace ringar
