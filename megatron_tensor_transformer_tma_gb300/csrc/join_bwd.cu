// Backward of the join on bf16 tensors.
#include "join_bwd.cuh"

namespace mlpb {

cudaError_t launch_join_bwd_bf16(const JoinParams& p, int grid, cudaStream_t s) {
  using bf = __nv_bfloat16;
  return p.post == MLPB_NORM_LAYER || p.pre == MLPB_NORM_LAYER
             ? join_bwd_pick<bf, bf, true>(p, grid, s)
             : join_bwd_pick<bf, bf, false>(p, grid, s);
}

}  // namespace mlpb
