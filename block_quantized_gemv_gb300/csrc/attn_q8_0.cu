// attn_q8_0.cu -- attention over a q8_0 cache: instantiations and launch.
#include "bqg_attn_launch.cuh"

namespace bqg {

cudaError_t attn_launch_q8_0(const AttnParams &p, int D, int rows, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    return attn_launch<BQG_Q8_0>(p, D, rows, plan, s, pdl);
}

}  // namespace bqg
