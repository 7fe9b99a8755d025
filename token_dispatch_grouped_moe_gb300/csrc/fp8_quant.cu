// fp8_quant.cu -- what makes the 8-bit operands of the expert products:
//   the residual's addition, the root-mean-square norm and its quantization
//     (launch_fp8_norm),
//   a weight's one-time quantization and transposition
//     (launch_fp8_quantize_weight),
//   the copy of quantized token rows into dispatch order (launch_fp8_dispatch).
// All are bound by memory: each value is read once and written once.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------ norm --
//
// One block per row; a thread holds VPT chunks of 8 consecutive columns in
// registers, so a row is read once. 16 neighbouring lanes hold one 128-column
// block, whose maximum is 4 shuffles away. Bound by memory from about a
// thousand rows on: 8192 rows of 4096 bf16 with residual move 303 MB in 48.2 us
// (6.3 TB/s, 0.94 of a plain copy's rate); one row is a launch and three trips
// to memory (2.5 us).

constexpr int kNormMaxThreads = 512;

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&o)[8])
{
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void load8(const __half* p, float (&o)[8])
{
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        o[2 * i] = f.x;
        o[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void load8(const float* p, float (&o)[8])
{
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}

template <typename T, int VPT>
__global__ void __launch_bounds__(kNormMaxThreads) fp8_norm_kernel(const Fp8NormArgs a)
{
    __shared__ float part[kNormMaxThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int n_vec = a.H / 8;
    const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + t * a.residual_stride : nullptr;
    float r[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < n_vec) {
            load8(x + 8 * v, r[i]);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) r[i][u] = 0.0f;
        }
    }
    if (res) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v < n_vec) {
                float b[8];
                load8(res + 8 * v, b);
#pragma unroll
                for (int u = 0; u < 8; ++u) r[i][u] += b[u];
            }
        }
    }
    if (a.sum) {
        T* sum = static_cast<T*>(a.sum) + t * a.sum_stride;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v < n_vec) store8(sum + 8 * v, r[i]);
        }
    }
    // the row's sum of squares (of the unrounded sums), in a fixed order
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int u = 0; u < 8; ++u) ss = fmaf(r[i][u], r[i][u], ss);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    float total = 0.0f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) total += part[w];
    const float inv_rms = 1.0f / sqrtf(total / (float)a.H + a.eps);

    const T* weight = static_cast<const T*>(a.weight);
    const int n_blocks = (a.H + kFp8Block - 1) / kFp8Block;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        const bool in = v < n_vec;
        float w8[8];
        if (weight && in) {
            load8(weight + 8 * v, w8);
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) w8[u] = 1.0f;
        }
        float amax = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            r[i][u] = r[i][u] * inv_rms * w8[u];
            if (in) amax = max_nan(amax, fabsf(r[i][u]));
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        if (!in) continue;
        if (a.y) store8(static_cast<T*>(a.y) + t * a.H + 8 * v, r[i]);
        const float scale = fp8_scale(amax);
        const float inv = 1.0f / scale;
        uint2 o;
        o.x = e4m3x4(r[i][0] * inv, r[i][1] * inv, r[i][2] * inv, r[i][3] * inv);
        o.y = e4m3x4(r[i][4] * inv, r[i][5] * inv, r[i][6] * inv, r[i][7] * inv);
        *reinterpret_cast<uint2*>(a.q + t * a.H + 8 * v) = o;
        if ((v & 15) == 0) a.scale[t * n_blocks + (v >> 4)] = scale;
    }
}

template <typename T>
cudaError_t launch_norm(const Fp8NormArgs& a, cudaStream_t s)
{
    const int n_vec = a.H / 8;
    const dim3 grid((unsigned)a.T);
    auto threads = [&](int vpt) { return dim3((unsigned)(((n_vec + vpt - 1) / vpt + 31) / 32 * 32)); };
    // one chunk a thread is the quickest for few rows; from 1024 rows on two
    // chunks of a 16-bit type (32 bytes in flight a thread and tensor, half the
    // threads to synchronise). Measured, one / two, us: H = 4096 with residual,
    // 1 row 2.5 / 2.8, 512: 4.6 / 5.1, 1024: 7.8 / 7.6, 8192: 57.5 / 48.2; H = 2048
    // without, 32768 rows 73.7 / 55.2; H = 512 (64 chunks) 34.2 / 35.1; fp32 (32
    // bytes a chunk), H = 4096, 8192 rows 84.9 / 85.4.
    const bool two = sizeof(T) == 2 && a.T >= 1024 && n_vec >= 128;
    if (n_vec <= kNormMaxThreads && !two) return launch_pdl(fp8_norm_kernel<T, 1>, grid, threads(1), 0, s, a);
    if (n_vec <= 2 * kNormMaxThreads) return launch_pdl(fp8_norm_kernel<T, 2>, grid, threads(2), 0, s, a);
    if (n_vec <= 4 * kNormMaxThreads) return launch_pdl(fp8_norm_kernel<T, 4>, grid, threads(4), 0, s, a);
    if (n_vec <= 8 * kNormMaxThreads) return launch_pdl(fp8_norm_kernel<T, 8>, grid, threads(8), 0, s, a);
    return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------- weight --
//
// One block per 128 x 128 block of one expert's weight [K, N]: read along N,
// kept in shared memory, written along K: 128 bytes of 4 rows a warp. Its reads
// of shared memory, 16 words of 4 columns and 8 places of K, lie in 4 banks (4-way
// conflicts); 32 rows of 16 bytes would have none and write half sectors. Made
// once for a weight: 64 experts 2048 x 1408 148 us, 3.7 TB/s, 0.56 of a copy.

constexpr int kWPitch = 130;   // 16-bit values per staged row of 128

__global__ void __launch_bounds__(256) fp8_quantize_weight_kernel(const uint16_t* __restrict__ w,
                                                                 uint8_t* __restrict__ q, float* __restrict__ scale,
                                                                 int K, int N)
{
    __shared__ uint16_t tile[kFp8Block * kWPitch];
    __shared__ float part[8];
    pdl_wait();
    pdl_launch_dependents();
    const int n0 = blockIdx.x * kFp8Block, k0 = blockIdx.y * kFp8Block;
    const int64_t e = blockIdx.z;
    const uint16_t* we = w + e * K * N;
    float amax = 0.0f;
    for (int c = threadIdx.x; c < kFp8Block * 16; c += 256) {   // chunks of 8 columns
        const int kk = c >> 4, nn = (c & 15) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k0 + kk < K && n0 + nn < N) v = *reinterpret_cast<const uint4*>(we + (int64_t)(k0 + kk) * N + n0 + nn);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<uint32_t*>(&tile[kk * kWPitch + nn + 2 * i]) = u[i];
            amax = max_nan(amax, max_nan(fabsf(__uint_as_float(u[i] << 16)), fabsf(__uint_as_float(u[i] & 0xffff0000u))));
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_nan(amax, part[i]);
    const float sc = fp8_scale(amax);
    if (threadIdx.x == 0)
        scale[(e * gridDim.x + blockIdx.x) * gridDim.y + blockIdx.y] = sc;
    for (int c = threadIdx.x; c < kFp8Block * 8; c += 256) {   // chunks of 16 k of one column
        const int nn = c >> 3, kk = (c & 7) * 16;
        if (n0 + nn >= N || k0 + kk >= K) continue;
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __uint_as_float((uint32_t)tile[(kk + i) * kWPitch + nn] << 16) / sc;
        *reinterpret_cast<uint4*>(q + (e * N + n0 + nn) * K + k0 + kk) =
            make_uint4(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]),
                       e4m3x4(f[8], f[9], f[10], f[11]), e4m3x4(f[12], f[13], f[14], f[15]));
    }
}

// -------------------------------------------------------------- dispatch --
//
// A warp per token: the token's row and scales are read once and written to
// each of its k dispatch positions.

__global__ void __launch_bounds__(256)
fp8_dispatch_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scale,
                    const int32_t* __restrict__ topk_idx, const int32_t* __restrict__ inv_pos,
                    const int32_t* __restrict__ r_valid, uint8_t* __restrict__ q_perm,
                    float* __restrict__ scale_perm, int64_t T, int32_t H, int32_t k, int32_t E, uint32_t* err)
{
    pdl_wait();
    pdl_launch_dependents();
    constexpr int U = 4;   // 16-byte words a lane holds: 2 KB of the row per pass
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    const int n_vec = H / 16;
    const int n_blocks = (H + kFp8Block - 1) / kFp8Block;
    const int64_t n_valid = *r_valid;
    for (int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < T; t += warps) {
        int p = -1;   // lane j < k: the position of the token's assignment j, or -1
        if (lane < k) {
            const int id = topk_idx[t * k + lane];
            if (id >= 0 && id < E) {
                p = inv_pos[t * k + lane];
                if (p < 0 || p >= n_valid) {
                    report_error(err, MOE_DEV_ERR_BOUNDS);
                    p = -1;
                }
            }
        }
        const uint4* src = reinterpret_cast<const uint4*>(q + t * H);
        for (int v0 = 0; v0 < n_vec; v0 += 32 * U) {
            uint4 r[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + 32 * u + lane < n_vec) r[u] = __ldg(src + v0 + 32 * u + lane);
            for (int j = 0; j < k; ++j) {
                const int pj = __shfl_sync(0xffffffffu, p, j);
                if (pj < 0) continue;
                uint4* dst = reinterpret_cast<uint4*>(q_perm + (int64_t)pj * H);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v0 + 32 * u + lane < n_vec) dst[v0 + 32 * u + lane] = r[u];
            }
        }
        for (int b0 = 0; b0 < n_blocks; b0 += 32) {
            const int b = b0 + lane;
            const float sc = b < n_blocks ? __ldg(scale + t * n_blocks + b) : 0.0f;
            for (int j = 0; j < k; ++j) {
                const int pj = __shfl_sync(0xffffffffu, p, j);
                if (pj >= 0 && b < n_blocks) scale_perm[(int64_t)pj * n_blocks + b] = sc;
            }
        }
    }
}

}  // namespace

cudaError_t launch_fp8_norm(moe_dtype dtype, const Fp8NormArgs& a, cudaStream_t s)
{
    if (a.T == 0) return cudaSuccess;
    switch (dtype) {
    case MOE_BF16: return launch_norm<__nv_bfloat16>(a, s);
    case MOE_FP16: return launch_norm<__half>(a, s);
    case MOE_FP32: return launch_norm<float>(a, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_fp8_quantize_weight(const uint16_t* w, uint8_t* q, float* scale, int32_t E, int32_t K, int32_t N,
                                       cudaStream_t s)
{
    const dim3 grid((N + kFp8Block - 1) / kFp8Block, (K + kFp8Block - 1) / kFp8Block, E);
    return launch_pdl(fp8_quantize_weight_kernel, grid, dim3(256), 0, s, w, q, scale, K, N);
}

cudaError_t launch_fp8_dispatch(const uint8_t* q, const float* scale, const int32_t* topk_idx, const int32_t* inv_pos,
                                const int32_t* r_valid, uint8_t* q_perm, float* scale_perm, int64_t T, int32_t H,
                                int32_t k, int32_t E, uint32_t* err, int num_sms, cudaStream_t s)
{
    if (T == 0) return cudaSuccess;
    const int64_t need = (T + 7) / 8;
    const int grid = (int)(need < (int64_t)num_sms * 8 ? need : (int64_t)num_sms * 8);
    return launch_pdl(fp8_dispatch_kernel, dim3(grid), dim3(256), 0, s, q, scale, topk_idx, inv_pos, r_valid, q_perm,
                      scale_perm, T, H, k, E, err);
}

}  // namespace moe
