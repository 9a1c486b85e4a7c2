// Instantiations of the scored attend (gqa_scored_kernel.cuh): bfloat16 caches.
#include "gqa_scored_kernel.cuh"

namespace gqa {

cudaError_t scored_bf16(int D, bool q_bf16, bool paged, const ScoredParams *p, cudaStream_t st, int *per_sm)
{
    return D == 128 ? scored::launch_d<kBf16, 128, false>(q_bf16, paged, p, st, per_sm)
                    : scored::launch_d<kBf16, 64, false>(q_bf16, paged, p, st, per_sm);
}

}  // namespace gqa
