// Cross attention: how a call is cut into blocks, and the join of gradients
// whose sums were split.
#include "attn_types.h"

namespace ringar {

// Blocks that keep the GPU busy: two a CU.  A call with fewer is split along
// what its blocks go along, down to parts of `least`.
static int splits_for(int64_t blocks, int64_t along, int64_t least) {
  const int64_t wanted = blocks ? 512 / blocks : 1, most = along / least;
  const int64_t s = wanted < most ? wanted : most;
  return s < 1 ? 1 : (int)s;
}

int64_t attn_blocks(const AttnArgs& a) { return (int64_t)a.tiles * a.splits * a.kv_heads * a.batch; }

void plan_attn_forward(int, AttnArgs& a) {
  a.few = a.rows <= 32;
  a.tiles = (int)(((int64_t)a.rows + (a.few ? 31 : 127)) / (a.few ? 32 : 128));
  a.splits = splits_for((int64_t)a.tiles * a.kv_heads * a.batch, a.keys, 256);
}

void plan_attn_dq(int, AttnArgs& a) {
  a.tiles = (int)(((int64_t)a.rows + 127) / 128);
  a.splits = splits_for((int64_t)a.tiles * a.kv_heads * a.batch, a.keys, 256);
}

void plan_attn_dkv(int, AttnArgs& a) {
  a.tiles = (int)(((int64_t)a.keys + 127) / 128);
  a.splits = splits_for((int64_t)a.tiles * a.kv_heads * a.batch, (int64_t)a.group * ((a.queries + 63) / 64), 2);
}

template <typename T> __global__ __launch_bounds__(256) void attn_join(AttnJoinArgs a) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < a.count; i += (int64_t)gridDim.x * 1024) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.splits; s++) {
      const Pack<float, 4> p = load_pack<float, 4>(a.part + s * a.apart + i);
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] += p.v[j];
    }
    Pack<T, 4> o;
#pragma unroll
    for (int j = 0; j < 4; j++) o.v[j] = (T)(v[j] * a.scale);
    store_pack<T, 4>((T*)a.out + i, o);
  }
}

hipError_t launch_attn_join(int dtype, const AttnJoinArgs& a, hipStream_t st) {
  const int64_t blocks = (a.count / 4 + 255) / 256;
  const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048));
  if (dtype == kF32) return launch_kernel(attn_join<float>, grid, 256, st, a);
  if (dtype == kF16) return launch_kernel(attn_join<_Float16>, grid, 256, st, a);
  return launch_kernel(attn_join<__bf16>, grid, 256, st, a);
}

#define RINGAR_BY_TYPE(call)                       \
  do {                                             \
    if (dtype == kF32) return call<float>(a, st);  \
    if (dtype == kF16) return call<_Float16>(a, st); \
    return call<__bf16>(a, st);                    \
  } while (0)

hipError_t launch_attn_forward(int dtype, const AttnArgs& a, hipStream_t st) { RINGAR_BY_TYPE(attn_forward_of); }
hipError_t launch_attn_delta(int dtype, const AttnArgs& a, hipStream_t st) { RINGAR_BY_TYPE(attn_delta_of); }
hipError_t launch_attn_dq(int dtype, const AttnArgs& a, hipStream_t st) { RINGAR_BY_TYPE(attn_dq_of); }
hipError_t launch_attn_dkv(int dtype, const AttnArgs& a, hipStream_t st) { RINGAR_BY_TYPE(attn_dkv_of); }

}  // namespace ringar
