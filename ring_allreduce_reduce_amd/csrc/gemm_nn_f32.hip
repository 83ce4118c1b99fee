// dx = dz weight: dz with k contiguous, weight with its columns contiguous (float).
#include "gemm_launch.h"

namespace ringar {
hipError_t launch_nn_f32(const GemmArgs& a, hipStream_t st) { return launch_tiled<float, true, false, kEpiStore>(a, st); }
}  // namespace ringar
