// The join between two blocks for a bf16 stream and bf16 blocks.
#include "join_bwd.cuh"
#include "join_fwd.cuh"

namespace mlpb {

template cudaError_t join_fwd_run<__nv_bfloat16, __nv_bfloat16>(const JoinParams&, int, cudaStream_t);
template cudaError_t join_bwd_run<__nv_bfloat16, __nv_bfloat16>(
    const JoinParams&, const JoinShape&, bool, int, cudaStream_t);

}  // namespace mlpb
