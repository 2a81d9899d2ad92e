// shared_bf16.cu -- attention behind shared tokens over a bf16 cache: instantiations and launch.
#include "bqg_attn_launch.cuh"

namespace bqg {

cudaError_t shared_launch_bf16(const SharedParams &p, int D, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    return shared_launch<BQG_BF16>(p, D, plan, s, pdl);
}

}  // namespace bqg
