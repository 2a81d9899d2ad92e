// attn_q4_0.cu -- attention over a q4_0 cache: instantiations and launch.
#include "bqg_attn_launch.cuh"

namespace bqg {

__device__ int g_attn_error_q4_0;

cudaError_t attn_launch_q4_0(const AttnParams &p, int D, int rows, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    return attn_launch<BQG_Q4_0>(p, D, rows, g_attn_error_q4_0, plan, s, pdl);
}
cudaError_t attn_take_error_q4_0(int *out) { return take_error(g_attn_error_q4_0, out); }

}  // namespace bqg
