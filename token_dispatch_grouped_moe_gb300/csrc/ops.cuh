// ops.cuh -- the launchers of routing from logits (route_logits.cuh), the
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

constexpr int kLinearBK = 64;        // K of a pipeline stage: one 128-byte swizzle span
constexpr int kLinearRowBox = 128;   // rows of a large and a small box of a
constexpr int kLinearRowBoxSmall = 32;

// Cut tiles of the product: their parts together hold at most kLinearPartRows rows
// of 128 fp32 sums in the workspace.
constexpr int kLinearMaxSplit = 16;
constexpr int kLinearMaxTickets = 512;
constexpr int kLinearPartRows = 81920;

// The kernel's forms: one CTA per MMA, tiles of 128 columns and up to 32 or 128 rows; a CTA
// pair per MMA, 256 columns and up to 256 or 128 rows.
enum LinearForm { kLinearFew = 0, kLinearOne = 1, kLinearPair = 2, kLinearPairHalf = 3 };
constexpr __host__ __device__ LinearForm linear_form_of(bool pair, int rows)
{
    return pair ? (rows == 256 ? kLinearPair : kLinearPairHalf) : (rows == 128 ? kLinearOne : kLinearFew);
}
inline __host__ __device__ bool linear_pair(LinearForm f) { return f >= kLinearPair; }
inline __host__ __device__ int linear_rows(LinearForm f) { return f == kLinearFew ? 32 : f == kLinearPair ? 256 : 128; }

// What the plan and the form are chosen by, in cycles. A K block (64) of a tile of r
// rows: shared memory passes the operands twice (128 bytes a cycle), 128 columns and r
// rows of one CTA, or r / 2 of each of a pair; that is more than the MMAs' own time for
// fewer than 256 rows of a pair, and for any of one CTA. Measured (cycles a block):
// pair, 256 rows 520; one CTA, 128 rows 480; a pair of 128 rows 380-460, and no less for
// fewer rows. Where every tile of the weights is read once, from memory, a CTA has no more
// than its stages in flight: 520, with nine of them instead of six 380.
constexpr float kLinearBytesPerCycle = 3580.0f;   // of the memory (6.8 TB/s at 1.9 GHz)
constexpr float kLinearL2Cycles = 80e6f / kLinearBytesPerCycle;   // of weights that L2 keeps beside the rows
inline __host__ __device__ float linear_block_cycles(LinearForm form, int rows, bool streamed)
{
    const float block = 256.0f + (linear_pair(form) ? 1.0f : 2.0f) * (float)rows;
    const float least = form == kLinearPairHalf ? 384.0f : streamed ? 520.0f : 0.0f;
    return block < least ? least : block;
}
// The last tile's epilogue, with nothing beside it.
constexpr float kLinearRowCycles = 16.0f;
// Publishing and joining the parts of a cut tile (measured: 128 rows in two parts on one
// CTA 10000 cycles, on a pair 9000, 256 on a pair 24000).
inline __host__ __device__ float linear_cut_cycles(LinearForm form, int rows, int parts, bool even)
{
    return (form == kLinearPair ? 1.5f : form == kLinearPairHalf ? 0.9f : 1.0f) *
           ((even ? 1.0f : 2.0f) * (2500.0f + 20.0f * (float)rows) + 1500.0f + 13.0f * (float)(rows * parts));
}
inline __host__ __device__ int linear_part_rows(int rows) { return (rows + 31) / 32 * 32; }

// A way to run `tiles` tiles of up to `rows` rows on n_units CTAs (or pairs): the first
// `full` whole, the K blocks of the rest in `segments` equal runs. Candidate 0: every
// tile whole; l: the tiles, where they fill less than one round, in l + 1 parts each;
// 31: the tiles beyond the whole rounds but one (or all of them) in equal runs. None
// is faster than the w_tiles different tiles of the weights come from memory: where
// they bound the product, the CTAs that have a tile of a round that is not full get the
// memory's whole rate, up to what a CTA has in flight. Cutting costs the parts'
// publication, twice where the runs do not line up with tiles, and the join's trips to L2.
struct LinearCandidate {
    bool fits;
    int full, segments;
    float cycles;
};
inline __host__ __device__ LinearCandidate linear_candidate(LinearForm form, int l, int tiles, int w_tiles, int rows,
                                                            int k_blocks, int n_units)
{
    const int cg = linear_pair(form) ? 2 : 1;
    const int rounds = (int)((unsigned)tiles / (unsigned)n_units), last = tiles - rounds * n_units;
    const float block = linear_block_cycles(form, rows, w_tiles == tiles);
    const float tile_bytes = (float)k_blocks * (float)(cg * 128 * kLinearBK * 2) * (1.0f / kLinearBytesPerCycle);
    float bytes = (float)w_tiles * tile_bytes;
    LinearCandidate c{l == 0, tiles, 0, 0.0f};
    if (l == 0) {
        const float whole = tiles ? bytes * ((float)(tiles - last) / (float)tiles) : 0.0f;
        const float run = (float)rounds * (float)k_blocks * block;
        c.cycles = run > whole ? run : whole;
        if (last) c.cycles += bytes - whole > (float)k_blocks * block ? bytes - whole : (float)k_blocks * block;
        c.cycles += kLinearRowCycles * (float)rows;
        return c;
    }
    // parts have room (and one more: a join reads up to 63 rows on), and the products of the
    // schedule stay below 2^32
    if (tiles == 0 || (2 * n_units * cg + 2) * linear_part_rows(rows) > kLinearPartRows || 2 * n_units * cg > kLinearMaxTickets ||
        k_blocks >= (1 << 30) / (n_units * n_units))
        return c;
    const bool even = l < 31;
    if (even ? rounds > 0 || l >= kLinearMaxSplit || tiles * (l + 1) > n_units : last == 0) return c;
    const int whole_rounds = !even && rounds > 1 ? rounds - 1 : 0;
    c.full = whole_rounds * n_units;
    c.segments = even ? tiles * (l + 1) : n_units;
    const unsigned left = (unsigned)(tiles - c.full);   // below 2 n_units
    const unsigned total = left * (unsigned)k_blocks;
    const int parts = even ? l + 1 : (int)((unsigned)n_units / left) + 2;
    c.fits = total >= 2u * (unsigned)c.segments;
    // runs that do not line up are at different places of K at a time: weights beyond L2 come
    // from memory again for each tile (700 x 14336 x 4096 in 128 rows: 109 us, now 76)
    if (!even && bytes > kLinearL2Cycles) bytes = (float)tiles * tile_bytes;
    const float run = ((float)(whole_rounds * k_blocks) + (float)total / (float)c.segments + 0.5f) * block;
    c.cycles = (run > bytes ? run : bytes) + linear_cut_cycles(form, rows, parts, even);
    return c;
}

// The candidate of the least cost: the lesser key (the cost's low bits give way to l).
inline __host__ __device__ uint32_t linear_candidate_key(const LinearCandidate& c, int l)
{
    union { float f; uint32_t u; } cycles = {c.cycles};
    return c.fits ? (cycles.u & ~31u) | (uint32_t)l : 0xffffffffu;
}
// The run (of `segments` equal ones over `total` K blocks) that holds a block.
inline __host__ __device__ int linear_segment_of(uint32_t block, uint32_t segments, uint32_t total)
{
    return (int)(((block + 1) * segments - 1) / total);
}

// The workspace of the product: the error word, the tiles' tickets (zero between
// calls), the parts.
constexpr size_t kLinearTicketOffset = 256;
constexpr size_t kLinearPartOffset = 256 + (size_t)kLinearMaxTickets * 4;
constexpr size_t kLinearWorkspaceBytes = kLinearPartOffset + (size_t)kLinearPartRows * 128 * 4;

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
    int32_t rows_per_warp;  // (set by the launcher)
};
// by the logits' type
cudaError_t launch_route_logits_bf16(const RouteLogitsArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_route_logits_fp16(const RouteLogitsArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_route_logits_fp32(const RouteLogitsArgs& a, int num_sms, cudaStream_t s);

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
cudaError_t launch_combine_rows(moe_dtype dtype, moe_dtype out_dtype, const CombineRowsArgs& a, cudaStream_t s);

}  // namespace moe
