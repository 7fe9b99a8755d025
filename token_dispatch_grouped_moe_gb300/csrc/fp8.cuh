// fp8.cuh -- what the 8-bit kernels share: block scales, e4m3 conversion
// (device), and the kernels' launchers (host). Internal.
//
// A value v of a block of 128 is held as e4m3 q with the block's fp32 scale:
//   scale = max(largest |v| of the block, 2^-100) / 448,
// q the nearest e4m3 (ties to even) to v / scale for weights and to v * (1 /
// scale) for activations, in fp32 (448 is the largest e4m3 value; the floor keeps
// the scale and its reciprocal finite for a block of zeros). A NaN in a block
// makes its scale and so the whole block NaN.
//
// The product with the reciprocal is within 2^-23 of the quotient, so q is another
// one for 2 of 10^7 values, whose quotients lie that near to the border between
// two: either is as near to v. The quotient costs activations a division, or two
// more FMAs a value: measured, us, 32768 x 2048 bf16 norm 54.7 -> 56.3, gated
// prefill of 64 experts 2048 -> 1408 1050 -> 1064.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"

namespace moe {

constexpr int kFp8Block = 128;        // values that share one scale
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxMin = 0x1p-100f;

// Cut tiles of the products (fp8_gemm.cu): their parts together hold at most
// kFp8PartRows rows of 256 fp32 sums in the workspace; costs in K blocks.
constexpr int kFp8MaxSplit = 16;
constexpr int kFp8MaxTickets = 512;
constexpr int kFp8PartRows = 40960;
constexpr float kFp8TileCost = 1.5f;
constexpr float kFp8CutCost = 7.0f;
constexpr float kFp8JoinCost = 1.4f;

// The workspace of the 8-bit products: the error word, the tiles' tickets
// (zero between calls), the parts.
constexpr size_t kFp8TicketOffset = 256;
constexpr size_t kFp8PartOffset = 256 + (size_t)kFp8MaxTickets * 4;
constexpr size_t kFp8WorkspaceBytes = kFp8PartOffset + (size_t)kFp8PartRows * 256 * 4;

enum Fp8GemmMode { kFp8Gated = 0, kFp8ProductBf16 = 1, kFp8ProductF32 = 2 };
// one CTA per MMA of 256 columns; of 128 (products only); a CTA pair per MMA
enum Fp8GemmForm { kFp8Wide = 0, kFp8Narrow = 1, kFp8Pair = 2 };

struct Fp8GemmArgs {
    int32_t R;                  // rows of A
    int32_t N;                  // output columns (gated: F)
    int32_t K;
    int32_t G;                  // groups (experts)
    const int32_t* offsets;     // [G+1], or null: one group of R rows
    const float* a_scale;       // [R, ceil(K/128)]
    const float* w0_scale;      // [G, ceil(N/128), ceil(K/128)]  (gated: of W1)
    const float* w1_scale;      // gated: of W3
    void* out;                  // gated: e4m3 [R, N]; product: bf16 or fp32 [R, N] or slot[k, T, N]
    float* out_scale;           // gated: [R, ceil(N/128)]
    const int32_t* src_row;     // product: scatter to slots, or null
    const float* topk_w;        // product with src_row: the gate weights by assignment
    int32_t k;
    int64_t T;
    int32_t* ticket;            // [kFp8MaxTickets], zero
    float* part;                // [kFp8PartRows, 256]
    uint32_t* err;
};

// tmA: A [R, K] e4m3, box 128 x 128; tmB0 / tmB1: weights [G, N, K] (gated: W1
// and W3; product: tmB1 unused), box 128 x fp8_box_rows; 128-byte swizzle.
inline uint32_t fp8_box_rows(bool gated, Fp8GemmForm form) { return gated ? 64 : form == kFp8Wide ? 256 : 128; }
cudaError_t launch_fp8_gemm(Fp8GemmMode mode, Fp8GemmForm form, const CUtensorMap& tmA, const CUtensorMap& tmB0,
                            const CUtensorMap& tmB1, const Fp8GemmArgs& a, int num_sms, cudaStream_t s);

struct Fp8NormArgs {
    const void* x;              // [T, H], rows x_stride elements apart
    const void* residual;       // or null
    const void* weight;         // [H] or null (ones)
    void* sum;                  // x + residual, rounded to the type, or null
    void* y;                    // [T, H] or null
    uint8_t* q;                 // [T, H] e4m3
    float* scale;               // [T, ceil(H/128)]
    int64_t T, x_stride, residual_stride, sum_stride;
    int32_t H;
    float eps;
};
cudaError_t launch_fp8_norm(moe_dtype dtype, const Fp8NormArgs& a, cudaStream_t s);

// w [E, K, N] bf16 -> q [E, N, K] e4m3 and the scales [E, ceil(N/128), ceil(K/128)] of its 128 x 128 blocks
cudaError_t launch_fp8_quantize_weight(const uint16_t* w, uint8_t* q, float* scale, int32_t E, int32_t K, int32_t N,
                                       cudaStream_t s);

// q_perm[p] = q[src_row[p] / k] and its scales, for the assignments with an id
// in [0, E), from the token side (each row read once)
cudaError_t launch_fp8_dispatch(const uint8_t* q, const float* scale, const int32_t* topk_idx, const int32_t* inv_pos,
                                const int32_t* r_valid, uint8_t* q_perm, float* scale_perm, int64_t T, int32_t H,
                                int32_t k, int32_t E, uint32_t* err, int num_sms, cudaStream_t s);

#ifdef __CUDACC__
// maximum that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float fp8_scale(float amax) { return max_nan(amax, kAmaxMin) / kE4m3Max; }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// x / (1 + e^-x); e^-x = inf for x below about -88 gives -0
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

__device__ __forceinline__ void store8(float* dst, const float (&o)[8])
{
    *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&o)[8])
{
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(bf16x2(o[0], o[1]), bf16x2(o[2], o[3]), bf16x2(o[4], o[5]), bf16x2(o[6], o[7]));
}

__device__ __forceinline__ void store4(float* dst, float a, float b, float c, float d)
{
    *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
}

__device__ __forceinline__ void store4(__nv_bfloat16* dst, float a, float b, float c, float d)
{
    *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2(a, b), bf16x2(c, d));
}

__device__ __forceinline__ uint32_t f16x2(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store8(__half* dst, const float (&o)[8])
{
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(f16x2(o[0], o[1]), f16x2(o[2], o[3]), f16x2(o[4], o[5]), f16x2(o[6], o[7]));
}
#endif

}  // namespace moe
