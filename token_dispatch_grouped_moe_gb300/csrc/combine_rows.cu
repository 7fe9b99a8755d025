// combine_rows.cu -- the weighted sum of experts' rows in token order:
//
//   out[t, :] = residual[t, :] + sum_j w[t, j] y[inv_pos[t, j], :]
//
// in fp32, the ranks j in order and the residual last, rounded once. A rank whose
// position lies outside [0, R) (an assignment that was dropped) adds nothing.
//
// Bound by memory: 32768 tokens' top 6 rows of 2048 bf16 with a residual 156 us for 1.08
// GB (6.9 TB/s, as a plain copy), 1531 tokens' top 8 of 3584 into fp32 20 us for 123 MB;
// one token 1.7 us, as any launch. A thread's k rows are loaded together (one after
// another: 176 and 23 us).
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "kernels.cuh"
#include "ops.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

// 8 values as they are in memory
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p)
{
    Eight<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    return r;
}

template <typename T>
__device__ __forceinline__ void floats_of(const Eight<T>& e, float (&f)[8])
{
    const uint32_t w[4] = {e.v[0].x, e.v[0].y, e.v[0].z, e.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            f[i] = __uint_as_float(w[i]);
        } else if constexpr (std::is_same<T, __half>::value) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    if constexpr (sizeof(T) == 4) {
        f[4] = __uint_as_float(e.v[1].x);
        f[5] = __uint_as_float(e.v[1].y);
        f[6] = __uint_as_float(e.v[1].z);
        f[7] = __uint_as_float(e.v[1].w);
    }
}

// A thread takes 8 columns of a token, all its rows' loads in flight together; a
// block `threads` such pieces of one token.
template <typename Y, typename OUT, int K>
__global__ void __launch_bounds__(256) combine_rows_kernel(const CombineRowsArgs a, unsigned pieces)
{
    pdl_wait();
    pdl_launch_dependents();
    const unsigned t = blockIdx.x / pieces;
    const int c = ((int)((blockIdx.x - t * pieces) * blockDim.x) + (int)threadIdx.x) * 8;
    if (c >= a.H) return;
    int32_t at[K];
    float w[K];
    bool there[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        at[j] = __ldg(a.inv_pos + (int64_t)t * K + j);
        w[j] = __ldg(a.topk_w + (int64_t)t * K + j);
    }
    Eight<OUT> res;
    if (a.residual) res = load8(static_cast<const OUT*>(a.residual) + t * a.residual_stride + c);
    // a dropped one's loads are of row 0, and not looked at: a branch between the loads
    // would make them wait for one another
    Eight<Y> v[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        there[j] = at[j] >= 0 && at[j] < a.R;
        v[j] = load8(static_cast<const Y*>(a.y) + (there[j] ? at[j] : 0) * a.y_stride + c);
    }
    float acc[8] = {}, f[8];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        floats_of<Y>(v[j], f);
        if (there[j]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
        }
    }
    if (a.residual) {
        floats_of<OUT>(res, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += f[i];
    }
    store8(static_cast<OUT*>(a.out) + t * a.out_stride + c, acc);
}

// No rows at all: the residual, or zeros.
template <typename OUT>
__global__ void __launch_bounds__(256) combine_nothing_kernel(const CombineRowsArgs a, unsigned pieces)
{
    pdl_wait();
    pdl_launch_dependents();
    const unsigned t = blockIdx.x / pieces;
    const int c = ((int)((blockIdx.x - t * pieces) * blockDim.x) + (int)threadIdx.x) * 8;
    if (c >= a.H) return;
    float f[8] = {};
    if (a.residual) floats_of<OUT>(load8(static_cast<const OUT*>(a.residual) + t * a.residual_stride + c), f);
    store8(static_cast<OUT*>(a.out) + t * a.out_stride + c, f);
}

template <typename Y, typename OUT>
cudaError_t launch(const CombineRowsArgs& a, cudaStream_t s)
{
    // blocks of one token's columns: all of them where 256 threads have them
    const int eights = a.H / 8;
    const unsigned threads = (unsigned)(eights >= 256 ? 256 : (eights + 31) / 32 * 32);
    const unsigned pieces = ((unsigned)eights + threads - 1) / threads;
    const dim3 grid((unsigned)a.T * pieces), block(threads);
    if (a.R == 0) return launch_pdl(combine_nothing_kernel<OUT>, grid, block, 0, s, a, pieces);
    switch (a.k) {
    case 1: return launch_pdl(combine_rows_kernel<Y, OUT, 1>, grid, block, 0, s, a, pieces);
    case 2: return launch_pdl(combine_rows_kernel<Y, OUT, 2>, grid, block, 0, s, a, pieces);
    case 3: return launch_pdl(combine_rows_kernel<Y, OUT, 3>, grid, block, 0, s, a, pieces);
    case 4: return launch_pdl(combine_rows_kernel<Y, OUT, 4>, grid, block, 0, s, a, pieces);
    case 5: return launch_pdl(combine_rows_kernel<Y, OUT, 5>, grid, block, 0, s, a, pieces);
    case 6: return launch_pdl(combine_rows_kernel<Y, OUT, 6>, grid, block, 0, s, a, pieces);
    case 7: return launch_pdl(combine_rows_kernel<Y, OUT, 7>, grid, block, 0, s, a, pieces);
    case 8: return launch_pdl(combine_rows_kernel<Y, OUT, 8>, grid, block, 0, s, a, pieces);
    }
    return cudaErrorInvalidValue;
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

cudaError_t launch_combine_rows(moe_dtype dtype, moe_dtype out_dtype, const CombineRowsArgs& a, cudaStream_t s)
{
    if (a.T == 0) return cudaSuccess;
    switch (dtype) {
    case MOE_BF16: return launch_out<__nv_bfloat16>(out_dtype, a, s);
    case MOE_FP16: return launch_out<__half>(out_dtype, a, s);
    case MOE_FP32: return launch_out<float>(out_dtype, a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
