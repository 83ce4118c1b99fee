// dx = dz weight: dz with k contiguous, weight with its columns contiguous (Float16).
#include "gemm_launch.h"

namespace ringar {
hipError_t launch_nn_f16(const GemmArgs& a, hipStream_t st) { return launch_tiled<_Float16, true, false, kEpiStore>(a, st); }
}  // namespace ringar
