// route_logits_fp32.cu -- routing from fp32 logits (route_logits.cuh).
#include "route_logits.cuh"

namespace moe {

cudaError_t launch_route_logits_fp32(const RouteLogitsArgs& a, int num_sms, cudaStream_t s)
{
    return launch_route_logits_of<float>(a, num_sms, s);
}

}  // namespace moe
