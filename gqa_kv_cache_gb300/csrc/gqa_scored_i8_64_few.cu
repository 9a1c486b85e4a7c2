// Instantiations of the scored attend (gqa_scored_kernel.cuh): 8-bit caches, D = 64, up to four query rows.
#include "gqa_scored_kernel.cuh"

namespace gqa {

cudaError_t scored_i8_64_few(bool q_bf16, bool paged, const ScoredParams *p, cudaStream_t st, int *per_sm)
{
    return scored::launch_d<kI8, 64, true, false>(q_bf16, paged, p, st, per_sm);
}

}  // namespace gqa
