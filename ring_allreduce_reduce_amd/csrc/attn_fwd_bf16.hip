#include "attn_forward.h"

namespace ringar {
template hipError_t attn_forward_of<__bf16>(const AttnArgs& a, hipStream_t st);
}
