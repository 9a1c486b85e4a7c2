// Instantiations of the scored attend (gqa_scored_kernel.cuh): 8-bit caches, D = 128, up to four query rows, capped, biased or counted scores.
#include "gqa_scored_kernel.cuh"

namespace gqa {

cudaError_t scored_i8_128_few_more(bool q_bf16, bool paged, const ScoredParams *p, cudaStream_t st, int *per_sm)
{
    return scored::launch_d<kI8, 128, true, true>(q_bf16, paged, p, st, per_sm);
}

}  // namespace gqa
