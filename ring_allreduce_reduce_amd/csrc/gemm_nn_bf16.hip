// dx = dz weight: dz with k contiguous, weight with its columns contiguous (bf16).
#include "gemm_launch.h"

namespace ringar {
hipError_t launch_nn_bf16(const GemmArgs& a, hipStream_t st) { return launch_tiled<__bf16, true, false, kEpiStore>(a, st); }
}  // namespace ringar
