// ops.cuh -- the launchers of routing from logits (route_logits.cu), the
// product with an epilogue (linear.cu) and the weighted sum of experts' rows
// (combine_rows.cu), and their arguments. Internal.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/moe.h"

namespace moe {

// ---------------------------------------------------------------- linear --

// Cut tiles of the product: their parts together hold at most kLinearPartRows rows
// of 128 fp32 sums in the workspace; costs in K blocks.
constexpr int kLinearMaxSplit = 16;
constexpr int kLinearMaxTickets = 512;
constexpr int kLinearPartRows = 81920;
constexpr float kLinearTileCost = 2.0f;
constexpr float kLinearCutCost = 4.0f;
constexpr float kLinearJoinCost = 0.05f;

// The workspace of the product: the error word, the tiles' tickets (zero between
// calls), the parts.
constexpr size_t kLinearTicketOffset = 256;
constexpr size_t kLinearPartOffset = 256 + (size_t)kLinearMaxTickets * 4;
constexpr size_t kLinearWorkspaceBytes = kLinearPartOffset + (size_t)kLinearPartRows * 128 * 4;

// one CTA per MMA, tiles of 128 columns and up to 128 rows; a CTA pair per MMA, 256 and 256
enum LinearForm { kLinearOne = 0, kLinearPair = 1 };

struct LinearArgs {
    int32_t R;                  // rows of a
    int32_t N;
    int32_t K;
    int32_t G;                  // groups (experts)
    const int32_t* offsets;     // [G+1], or null: one group of R rows
    const void* bias;           // [G, N] or null
    int32_t bias_f32;           // its type: fp32, or the operands'
    int32_t act;                // moe_activation
    const void* residual;       // out's type, or null; rows residual_stride elements apart
    int64_t residual_stride;
    void* out;
    int64_t out_stride;
    int32_t fp16;               // operands: fp16, or bf16
    int32_t w_nk;               // the weights' layout: [G, N, K], or [G, K, N]
    int32_t tile_rows;          // rows of a tile at most
    int32_t* ticket;            // [kLinearMaxTickets], zero
    float* part;                // [kLinearPartRows, 128]
    uint32_t* err;
};

constexpr int kLinearBK = 64;        // K of a pipeline stage: one 128-byte swizzle span
constexpr int kLinearRowBox = 128;   // rows of a large and a small box of a
constexpr int kLinearRowBoxSmall = 32;

// tm_a / tm_a_small: a [R, K], boxes of 64 values x 128 / 32 rows; tm_w: [G, K, N],
// box 64 n x 64 k, or [G, N, K], box 64 k x 128 n. 128-byte swizzle.
cudaError_t launch_linear(LinearForm form, moe_dtype out_dtype, const CUtensorMap& tm_a, const CUtensorMap& tm_a_small,
                          const CUtensorMap& tm_w, const LinearArgs& a, int num_sms, cudaStream_t s);

// A TMA tensor map of 16-bit values, dims innermost first (rank 2 or 3, strides
// in bytes of the outer ones), a 128-byte swizzle; elements outside read as zero.
bool encode_map_b16(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                    const uint32_t* box);

// ---------------------------------------------------------- route_logits --

struct RouteLogitsArgs {
    const void* logits;     // [T, E], rows `stride` elements apart
    int64_t stride;
    const float* bias;      // [E] or null
    int32_t* topk_idx;      // [T, k]
    float* topk_w;          // [T, k]
    int64_t T;
    int32_t E, k;
    int32_t sigmoid;        // scores: sigmoid, or softmax
    int32_t groups, top_groups, group_top;
    int32_t renorm;
    float scale;
};
cudaError_t launch_route_logits(moe_dtype dtype, const RouteLogitsArgs& a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------- combine_rows --

struct CombineRowsArgs {
    const void* y;              // [R, H], rows y_stride elements apart
    const int32_t* inv_pos;     // [T, k]
    const float* topk_w;        // [T, k]
    const void* residual;       // [T, H] of the output's type, or null
    void* out;                  // [T, H]
    int64_t T, R, y_stride, residual_stride, out_stride;
    int32_t H, k;
};
cudaError_t launch_combine_rows(moe_dtype dtype, moe_dtype out_dtype, const CombineRowsArgs& a, int num_sms,
                                cudaStream_t s);

}  // namespace moe
