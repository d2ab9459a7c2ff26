// gdn_attn_sparse_forward over a cache in 8 or 4 bits.
#include "gdn_attn_tile.h"

namespace gdn {

hipError_t launch_attn_sparse_coded(const SparseArgs& p, void* workspace, hipStream_t stream) {
  return p.cache.format == kCacheE4M3 ? launch_attn_f<kE4M3, true>(p, workspace, stream)
                                      : launch_attn_f<kE2M1, true>(p, workspace, stream);
}

}  // namespace gdn
