// The tensor-core kernels of linear attention for bf16 rows.
#include "state_chunk.cuh"

namespace sv {

cudaError_t launch_state_chunk_bf16(const StateChunkPlan &A, bool outputs, const CUtensorMap *maps, cudaStream_t st) {
  constexpr int DT = SPEC_DTYPE_BF16;
  if (A.p.key_dim <= 64) return outputs ? launch_chunks<DT, 64, true>(A, maps, st) : launch_chunks<DT, 64, false>(A, maps, st);
  return outputs ? launch_chunks<DT, 128, true>(A, maps, st) : launch_chunks<DT, 128, false>(A, maps, st);
}

cudaError_t launch_state_short_bf16(const StateChunkPlan &A, const CUtensorMap *maps, cudaStream_t st) {
  constexpr int DT = SPEC_DTYPE_BF16;
  return A.p.key_dim <= 64 ? launch_short<DT, 64>(A, maps, st) : launch_short<DT, 128>(A, maps, st);
}

}  // namespace sv
