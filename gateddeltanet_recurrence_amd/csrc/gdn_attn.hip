// gdn_attn_forward over a cache in the I/O type or in 8 bits.
#include "gdn_attn_tile.h"

namespace gdn {

hipError_t launch_attn(const AttnArgs& p, int io_dtype, void* workspace, hipStream_t stream) {
  if (p.rows.N == 0) return hipSuccess;
  if (io_dtype != 1) return launch_attn_f<kF32, false>(p, workspace, stream);
  if (p.cache.format == kCacheE2M1) return launch_attn_e2m1(p, workspace, stream);
  return p.cache.format == kCacheE4M3 ? launch_attn_f<kE4M3, false>(p, workspace, stream)
                                      : launch_attn_f<kF16, false>(p, workspace, stream);
}

size_t attn_workspace_bytes(int64_t N, int64_t R, int Hq, int Hk, int D, int format) {
  if (N == 0 || R == 0) return 0;
  const int rows = part_rows(N, Hq / Hk);
  if (format == kCacheE2M1) return kNoteBytes4 + (size_t)2 * kMostGroups4 * rows * (D + 2) * sizeof(float);
  return kNoteBytes + (size_t)2 * (D == 64 ? kMostGroups : kGroups) * rows * (D + 2) * sizeof(float);
}

}  // namespace gdn
