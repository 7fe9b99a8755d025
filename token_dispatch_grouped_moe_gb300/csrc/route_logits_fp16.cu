// route_logits_fp16.cu -- routing from fp16 logits (route_logits.cuh).
#include "route_logits.cuh"

namespace moe {

cudaError_t launch_route_logits_fp16(const RouteLogitsArgs& a, int num_sms, cudaStream_t s)
{
    return launch_route_logits_of<__half>(a, num_sms, s);
}

}  // namespace moe
