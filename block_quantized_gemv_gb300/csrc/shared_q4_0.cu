// shared_q4_0.cu -- attention behind shared tokens over a q4_0 cache: instantiations and launch.
#include "bqg_attn_launch.cuh"

namespace bqg {

cudaError_t shared_launch_q4_0(const SharedParams &p, int D, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    return shared_launch<BQG_Q4_0>(p, D, plan, s, pdl);
}

}  // namespace bqg
