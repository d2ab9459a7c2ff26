// gdn_attn_forward over a cache in 4 bits.
#include "gdn_attn_tile.h"

namespace gdn {

hipError_t launch_attn_e2m1(const AttnArgs& p, void* workspace, hipStream_t stream) {
  return launch_attn_f<kE2M1, false>(p, workspace, stream);
}

}  // namespace gdn
