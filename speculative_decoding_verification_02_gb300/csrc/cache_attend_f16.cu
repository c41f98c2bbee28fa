// spec_cache_attend's tensor-core kernels for fp16 rows.
#include "cache_attend_tile.cuh"

namespace sv {

cudaError_t launch_cache_attend_f16(const CacheTilePlan &A, const CUtensorMap &map, int copies, cudaStream_t st) {
  return A.p.c.head_dim == 128 ? launch_tiles<SPEC_DTYPE_F16, 128>(A, map, copies, st) : launch_tiles<SPEC_DTYPE_F16, 64>(A, map, copies, st);
}

}  // namespace sv
