// attn_bf16.cu -- attention over a bf16 cache: instantiations and launch.
#include "bqg_attn_launch.cuh"

namespace bqg {

cudaError_t attn_launch_bf16(const AttnParams &p, int D, int rows, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    return attn_launch<BQG_BF16>(p, D, rows, plan, s, pdl);
}

}  // namespace bqg
