#include "attn_backward.h"

namespace ringar {
template hipError_t attn_delta_of<float>(const AttnArgs& a, hipStream_t st);
template hipError_t attn_dq_of<float>(const AttnArgs& a, hipStream_t st);
template hipError_t attn_dkv_of<float>(const AttnArgs& a, hipStream_t st);
}
