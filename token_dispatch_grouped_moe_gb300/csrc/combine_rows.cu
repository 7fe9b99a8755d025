// combine_rows.cu -- the weighted sum of experts' rows in token order:
//
//   out[t, :] = residual[t, :] + sum_j w[t, j] y[inv_pos[t, j], :]
//
// in fp32, the ranks j in order and the residual last, rounded once. A rank whose
// position lies outside [0, R) (an assignment that was dropped) adds nothing.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "kernels.cuh"
#include "ops.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void load8(const float* p, float (&v)[8])
{
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8])
{
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void load8(const __half* p, float (&v)[8])
{
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// a block takes 8 * kThreads columns of one token, a thread 8 of them
template <typename Y, typename OUT>
__global__ void __launch_bounds__(kThreads) combine_rows_kernel(const CombineRowsArgs a, int pieces)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x / (unsigned)pieces;
    const int c = ((int)(blockIdx.x % (unsigned)pieces) * kThreads + (int)threadIdx.x) * 8;
    if (c >= a.H) return;
    float acc[8] = {};
    for (int j = 0; j < a.k; ++j) {
        const int32_t p = __ldg(a.inv_pos + t * a.k + j);
        if (p < 0 || p >= a.R) continue;
        const float w = __ldg(a.topk_w + t * a.k + j);
        float v[8];
        load8(static_cast<const Y*>(a.y) + p * a.y_stride + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
    }
    if (a.residual) {
        float v[8];
        load8(static_cast<const OUT*>(a.residual) + t * a.residual_stride + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
    store8(static_cast<OUT*>(a.out) + t * a.out_stride + c, acc);
}

template <typename Y, typename OUT>
cudaError_t launch(const CombineRowsArgs& a, cudaStream_t s)
{
    const int pieces = (a.H / 8 + kThreads - 1) / kThreads;
    return launch_pdl(combine_rows_kernel<Y, OUT>, dim3((unsigned)(a.T * pieces)), dim3(kThreads), 0, s, a, pieces);
}

template <typename Y>
cudaError_t launch_out(moe_dtype out, const CombineRowsArgs& a, cudaStream_t s)
{
    switch (out) {
    case MOE_BF16: return launch<Y, __nv_bfloat16>(a, s);
    case MOE_FP16: return launch<Y, __half>(a, s);
    case MOE_FP32: return launch<Y, float>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_combine_rows(moe_dtype dtype, moe_dtype out_dtype, const CombineRowsArgs& a, int num_sms,
                                cudaStream_t s)
{
    (void)num_sms;
    if (a.T == 0) return cudaSuccess;
    switch (dtype) {
    case MOE_BF16: return launch_out<__nv_bfloat16>(out_dtype, a, s);
    case MOE_FP16: return launch_out<__half>(out_dtype, a, s);
    case MOE_FP32: return launch_out<float>(out_dtype, a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
