// attn_bf16.cu -- attention over a bf16 cache: instantiations and launch.
#include "bqg_attn_launch.cuh"

namespace bqg {

__device__ int g_attn_error_bf16;

cudaError_t attn_launch_bf16(const AttnParams &p, int D, int rows, AttnPlan *plan, cudaStream_t s, bool pdl)
{
    return attn_launch<BQG_BF16>(p, D, rows, g_attn_error_bf16, plan, s, pdl);
}
cudaError_t attn_take_error_bf16(int *out) { return take_error(g_attn_error_bf16, out); }

}  // namespace bqg
