// route_logits_bf16.cu -- routing from bf16 logits (route_logits.cuh).
#include "route_logits.cuh"

namespace moe {

cudaError_t launch_route_logits_bf16(const RouteLogitsArgs& a, int num_sms, cudaStream_t s)
{
    return launch_route_logits_of<__nv_bfloat16>(a, num_sms, s);
}

}  // namespace moe
