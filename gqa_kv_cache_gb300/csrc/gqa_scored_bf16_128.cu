// Instantiations of the scored attend (gqa_scored_kernel.cuh): bfloat16 caches, D = 128.
#include "gqa_scored_kernel.cuh"

namespace gqa {

cudaError_t scored_bf16_128(bool q_bf16, bool paged, const ScoredParams *p, cudaStream_t st, int *per_sm)
{
    return scored::launch_d<kBf16, 128, false, true>(q_bf16, paged, p, st, per_sm);
}

}  // namespace gqa
