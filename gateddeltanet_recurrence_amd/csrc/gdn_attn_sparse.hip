// gdn_attn_sparse_forward over a cache in the I/O type.
#include "gdn_attn_tile.h"

namespace gdn {

hipError_t launch_attn_sparse(const SparseArgs& p, int io_dtype, void* workspace, hipStream_t stream) {
  if (p.rows.N == 0) return hipSuccess;
  if (io_dtype != 1) return launch_attn_f<kF32, true>(p, workspace, stream);
  return p.cache.format == kCacheIo ? launch_attn_f<kF16, true>(p, workspace, stream)
                                    : launch_attn_sparse_coded(p, workspace, stream);
}

}  // namespace gdn
