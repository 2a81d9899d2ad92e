// attn_q4_0.cu -- attention over a q4_0 cache: instantiations and launch.
#include "bqg_attn_launch.cuh"

namespace bqg {

cudaError_t attn_launch_q4_0(const AttnParams &p, int D, int rows, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    return attn_launch<BQG_Q4_0>(p, D, rows, plan, s, pdl);
}

}  // namespace bqg
