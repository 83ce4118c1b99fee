#include "attn_forward.h"

namespace ringar {
template hipError_t attn_forward_of<float>(const AttnArgs& a, hipStream_t st);
}
