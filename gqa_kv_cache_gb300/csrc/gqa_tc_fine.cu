// Tensor-core decode kernel, the form with the weights in three bfloat16 parts
// (attend over selected blocks of a bfloat16 cache).
#define GQA_MULTI_TOKEN 0
#include "gqa_tc_kernel.cuh"

namespace gqa {

cudaError_t tc_launch_fine(const DecodeParams &p, const TcMaps &maps, cudaStream_t st)
{
    return p.q_bf16 ? launch_q<false, false, false, false, 0, true>(p, maps, st)
                    : launch_q<true, false, false, false, 0, true>(p, maps, st);
}

}  // namespace gqa
