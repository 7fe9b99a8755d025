// api_ops.cu -- the C ABI of moe_route_logits, moe_linear and moe_combine_rows
// (include/moe.h): argument checks, TMA descriptors and launches. Host code only.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe.h"
#include "api.h"
#include "kernels.cuh"
#include "ops.cuh"

namespace moe {
namespace {

constexpr int32_t kMaxTopK = 8;
constexpr int32_t kMaxExperts = 256;
constexpr int32_t kMaxGroupsOfExperts = 32;

static_assert(kLinearPartOffset == MOE_LINEAR_WORKSPACE_ZEROS, "what has to be zero lies before the parts");

bool is_dtype(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_FP32; }
int size_of(moe_dtype t) { return t == MOE_FP32 ? 4 : 2; }
// The sizes of a product: R rows, G weights of [K, N] (a copy's rows of contiguous values, n
// or k, are 16 bytes apart).
moe_status check_linear(int64_t R, int32_t K, int32_t N, int32_t G, moe_weight_layout layout)
{
    if (R < 0 || K <= 0 || N <= 0 || G <= 0) return MOE_ERR_INVALID_ARG;
    if (K % 8 || (layout == MOE_WEIGHT_KN && N % 8) || K > (1 << 30) || N > (1 << 30) || G > kMaxExperts || R >= ((int64_t)1 << 31) - 256)
        return MOE_ERR_UNSUPPORTED;
    // tiles, and a round of them more, are counted in 32 bits
    if ((R / 128 + G) * (((int64_t)N + 127) / 128) >= ((int64_t)1 << 31) - (1 << 16)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// The estimated cycles of a product in tiles of up to `cap` rows, for groups of equal size.
float linear_cycles(LinearForm form, int64_t R, int32_t K, int32_t N, int32_t G, int sms)
{
    const bool pair = linear_pair(form);
    const int cap = linear_rows(form), step = pair ? 32 : 16, cols = pair ? 256 : 128, units = pair ? sms / 2 : sms;
    if (units <= 0) return INFINITY;
    const int64_t active = R < G ? R : G, rows = (R + active - 1) / active;
    const int64_t m_tiles = (rows + cap - 1) / cap, n_tiles = ((int64_t)N + cols - 1) / cols;
    const int per = (int)(((rows + m_tiles - 1) / m_tiles + step - 1) / step * step);
    const int64_t tiles = active * m_tiles * n_tiles;
    if (tiles >= ((int64_t)1 << 31)) return INFINITY;
    float best = INFINITY;
    for (int l = 0; l < 32; ++l) {
        const LinearCandidate c = linear_candidate(form, l, (int)tiles, (int)(active * n_tiles), per,
                                                   (K + kLinearBK - 1) / kLinearBK, units);
        if (c.fits && c.cycles < best) best = c.cycles;
    }
    return best;
}

// The form of a product over R rows in G groups: a pair where its estimate is less by a
// thirtieth at least, in the pairs' two heights the lesser; few rows in the form that
// leaves room for the next kernel's CTA.
// Measured, one CTA / pair of 256 rows / pair of 128, us, K x N: 4096 x 256, 8192 rows 21.9 / 24.5 /
// 19.2; 4096 x 1024, 2000 21.4 / 24.3 / 18.7, 4096 36.4 / 27.5 / 29.2; 1024 x 4096, 400 10.1 / 10.8
// / 10.1, 700 13.4 / 12.6 / 11.7; 4096 x 4096, 256 17.8 / 23.7 / 16.3, 400 21.0 / 22.0 / 18.2, 700
// 31.8 / 25.5 / 29.4, 8192 219 / 147 / 175; 4096 x 14336, 100 25.2 / 26.7 / 23.9, 160 35.6 / 27.8 /
// 30.1; 14336 x 4096, 160 38.5 / 41.7 / 32.5, 256 41.1 / 47.2 / 34.9; 8192 x 8192, 256 37.8 / 41.8 /
// 32.0, 400 65.2 / 41.6 / 50.6; 8192 x 512, 400 17.8 / 25.0 / 16.6; 2048 x 128, 100 12.1 / 11.7 /
// 10.0; 64 groups 2048 x 1408, 50 each 64.1 / 71.4 / 69.7, 128 70.0 / 75.1 / 72.2, 180 95.7 / 80.1 /
// 85.8. The form taken is 0.7% off the best of the three on average over 187 such sizes, 10% at worst
// (400 x 14336 x 4096 49.0 for 44.5). Up to 32 / 128 rows, one CTA: 1 row 4096 x 14336 23.5 / 24.1,
// 8 rows 4096 x 4096 9.5 / 10.4, 14336 x 4096 24.0 / 23.7, 32 rows 1024 x 4096 8.3 / 7.1.
LinearForm linear_form(int64_t R, int32_t K, int32_t N, int32_t G, int sms)
{
    if (G == 1 && R <= 16) return kLinearFew;
    const float one = linear_cycles(kLinearOne, R, K, N, G, sms);
    const float pair = linear_cycles(kLinearPair, R, K, N, G, sms) * (30.0f / 29.0f);
    const float half = linear_cycles(kLinearPairHalf, R, K, N, G, sms);
    if (one <= pair && one <= half) return kLinearOne;
    return pair <= half ? kLinearPair : kLinearPairHalf;
}

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_logits(int64_t T, int32_t E, int32_t k, moe_dtype dtype, const void* logits, int64_t stride,
                            const moe_scoring* scoring, int32_t* topk_idx, float* topk_w, moe_stream_t stream)
{
    const moe_scoring plain{MOE_SCORES_SOFTMAX, nullptr, 1, 1, 1, 0, 1.0f};
    const moe_scoring& c = scoring ? *scoring : plain;
    if (T < 0 || E <= 0 || k <= 0 || k > E) return MOE_ERR_INVALID_ARG;
    if (c.scores != MOE_SCORES_SOFTMAX && c.scores != MOE_SCORES_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (c.groups <= 0 || E % c.groups || c.top_groups <= 0 || c.top_groups > c.groups) return MOE_ERR_INVALID_ARG;
    if ((c.group_top != 1 && c.group_top != 2) || c.group_top > E / c.groups) return MOE_ERR_INVALID_ARG;
    if (k > c.top_groups * (E / c.groups) || !std::isfinite(c.scale)) return MOE_ERR_INVALID_ARG;
    if (!is_dtype(dtype) || k > kMaxTopK || E > kMaxExperts || c.groups > kMaxGroupsOfExperts) return MOE_ERR_UNSUPPORTED;
    if (T >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!logits || !topk_idx || !topk_w || (T > 1 && stride < E)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(logits, size_of(dtype)) || !aligned_to(c.bias, 4) || !aligned_to(topk_idx, 4) ||
        !aligned_to(topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    const int sms = num_sms_current();
    if (sms <= 0) return MOE_ERR_CUDA;
    Range range("moe/route_logits");
    const RouteLogitsArgs a{logits, stride, c.bias, topk_idx, topk_w, T, E, k, c.scores == MOE_SCORES_SIGMOID,
                            c.groups, c.top_groups, c.group_top, c.renormalize != 0, c.scale, 1};
    const auto launch = dtype == MOE_BF16 ? launch_route_logits_bf16
                        : dtype == MOE_FP16 ? launch_route_logits_fp16
                                            : launch_route_logits_fp32;
    return finish(launch(a, sms, (cudaStream_t)stream), nullptr, (cudaStream_t)stream);
}

size_t moe_linear_workspace_size(void) { return kLinearWorkspaceBytes; }

moe_status moe_linear(int64_t R, int32_t K, int32_t N, int32_t G, moe_dtype dtype, const void* a, int64_t a_stride,
                      const int32_t* offsets, const void* w, moe_weight_layout layout, const moe_epilogue* epilogue,
                      moe_dtype out_dtype, void* out, int64_t out_stride, void* ws, size_t ws_bytes,
                      moe_stream_t stream)
{
    const moe_epilogue plain{nullptr, MOE_FP32, MOE_ACT_NONE, nullptr, 0};
    const moe_epilogue& e = epilogue ? *epilogue : plain;
    if (R < 0 || K <= 0 || N <= 0 || G <= 0 || (!offsets && G != 1)) return MOE_ERR_INVALID_ARG;
    if (layout != MOE_WEIGHT_KN && layout != MOE_WEIGHT_NK) return MOE_ERR_INVALID_ARG;
    if (e.activation < MOE_ACT_NONE || e.activation > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_BF16 && dtype != MOE_FP16) return MOE_ERR_UNSUPPORTED;
    if (out_dtype != dtype && out_dtype != MOE_FP32) return MOE_ERR_UNSUPPORTED;
    if (e.bias && e.bias_dtype != dtype && e.bias_dtype != MOE_FP32) return MOE_ERR_UNSUPPORTED;
    MOE_TRY_STATUS(check_linear(R, K, N, G, layout));
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < kLinearWorkspaceBytes) return MOE_ERR_WORKSPACE;
    if (R == 0) return MOE_OK;
    if (!a || !w || !out || !aligned16(a) || !aligned16(w)) return MOE_ERR_INVALID_ARG;
    if (R > 1 && (a_stride < K || a_stride % 8 || out_stride < N || (e.residual && e.residual_stride < N)))
        return MOE_ERR_INVALID_ARG;
    if (!aligned_to(out, size_of(out_dtype)) || !aligned_to(e.residual, size_of(out_dtype)) ||
        (e.bias && !aligned_to(e.bias, size_of(e.bias_dtype))) || !aligned_to(offsets, 4))
        return MOE_ERR_INVALID_ARG;
    const int sms = num_sms_current();
    if (sms <= 0) return MOE_ERR_CUDA;
    Range range("moe/linear");
    if (R == 1) a_stride = K;
    const bool nk = layout == MOE_WEIGHT_NK;
    const uint64_t a_dims[] = {(uint64_t)K, (uint64_t)R}, a_strides[] = {(uint64_t)a_stride * 2};
    const uint32_t large[] = {kLinearBK, kLinearRowBox}, small[] = {kLinearBK, kLinearRowBoxSmall};
    const uint64_t inner = nk ? K : N, outer = nk ? N : K;
    const uint64_t w_dims[] = {inner, outer, (uint64_t)G}, w_strides[] = {inner * 2, inner * outer * 2};
    const uint32_t w_box[] = {64, nk ? 128u : 64u, 1};
    CUtensorMap tm_a, tm_a_small, tm_w;
    if (!encode_map_b16(&tm_a, a, 2, a_dims, a_strides, large) || !encode_map_b16(&tm_a_small, a, 2, a_dims, a_strides, small) ||
        !encode_map_b16(&tm_w, w, 3, w_dims, w_strides, w_box))
        return MOE_ERR_CUDA;
    LinearArgs args{};
    args.R = (int32_t)R;
    args.N = N;
    args.K = K;
    args.G = G;
    args.offsets = offsets;
    args.bias = e.bias;
    args.bias_f32 = e.bias_dtype == MOE_FP32;
    args.act = e.activation;
    args.residual = e.residual;
    args.residual_stride = e.residual_stride;
    args.out = out;
    args.out_stride = out_stride;
    args.fp16 = dtype == MOE_FP16;
    args.w_nk = nk;
    unsigned char* b = static_cast<unsigned char*>(ws);
    args.ticket = reinterpret_cast<int32_t*>(b + kLinearTicketOffset);
    args.part = reinterpret_cast<float*>(b + kLinearPartOffset);
    args.err = static_cast<uint32_t*>(ws);
    const LinearForm form = linear_form(R, K, N, G, sms);
    args.tile_rows = linear_rows(form);
    return finish(launch_linear(form, out_dtype, tm_a, tm_a_small, tm_w, args, sms, (cudaStream_t)stream), ws,
                  (cudaStream_t)stream);
}

int32_t moe_selftest_linear_form(int64_t R, int32_t K, int32_t N, int32_t G, int32_t num_sms)
{
    if (check_linear(R, K, N, G, MOE_WEIGHT_KN) != MOE_OK || R == 0 || num_sms <= 0) return -1;
    return linear_form(R, K, N, G, num_sms);
}

moe_status moe_selftest_linear_schedule(int64_t R, int32_t K, int32_t N, int32_t G, const int32_t* offsets,
                                        int32_t num_sms, moe_linear_schedule* schedule)
{
    if (!schedule || num_sms <= 0 || (!offsets && G != 1)) return MOE_ERR_INVALID_ARG;
    MOE_TRY_STATUS(check_linear(R, K, N, G, MOE_WEIGHT_NK));
    *schedule = moe_linear_schedule{};
    if (R == 0) return MOE_OK;   // nothing is launched
    const LinearForm form = linear_form(R, K, N, G, num_sms);
    const bool pair = linear_pair(form);
    const int step = pair ? 32 : 16, cap = linear_rows(form), units = pair ? num_sms / 2 : num_sms;
    const int n_tiles = (int)(((int64_t)N + (pair ? 255 : 127)) / (pair ? 256 : 128));
    const int k_blocks = (K + kLinearBK - 1) / kLinearBK;
    int row_tiles = 0, most = 0, groups = 0;
    for (int g = 0; g < G; ++g) {
        const int64_t lo = offsets ? offsets[g] : 0, hi = offsets ? offsets[g + 1] : R;
        if (lo < 0 || hi < lo || hi > R) return MOE_ERR_INVALID_ARG;
        if (hi == lo) continue;
        const int rows = (int)(hi - lo), tiles = (int)((hi - lo + cap - 1) / cap);
        const int per = (int)(((int64_t)rows + tiles - 1) / tiles + step - 1) / step * step;
        most = per > most ? per : most;
        row_tiles += tiles;
        ++groups;
    }
    const int tiles = row_tiles * n_tiles;
    LinearCandidate best{};
    uint32_t least = 0xffffffffu;
    for (int l = 0; l < 32; ++l) {
        const LinearCandidate c = linear_candidate(form, l, tiles, groups * n_tiles, most, k_blocks, units);
        const uint32_t key = linear_candidate_key(c, l);
        if (key < least) { least = key; best = c; }
    }
    *schedule = moe_linear_schedule{form, units, tiles, best.full, best.segments, linear_part_rows(most), 0};
    const uint32_t total = (uint32_t)(tiles - best.full) * (uint32_t)k_blocks, runs = (uint32_t)best.segments;
    for (int q = 0; runs && q < tiles - best.full; ++q) {
        const int parts = linear_segment_of((uint32_t)(q + 1) * (uint32_t)k_blocks - 1, runs, total) -
                          linear_segment_of((uint32_t)q * (uint32_t)k_blocks, runs, total) + 1;
        if (parts > schedule->most_parts) schedule->most_parts = parts;
    }
    return MOE_OK;
}

moe_status moe_combine_rows(int64_t T, int32_t H, int32_t k, int64_t R, moe_dtype dtype, const void* y,
                            int64_t y_stride, const int32_t* inv_pos, const float* topk_w, moe_dtype out_dtype,
                            const void* residual, int64_t residual_stride, void* out, int64_t out_stride,
                            moe_stream_t stream)
{
    if (T < 0 || H <= 0 || k <= 0 || R < 0) return MOE_ERR_INVALID_ARG;
    if (!is_dtype(dtype) || !is_dtype(out_dtype) || H % 8 || k > kMaxTopK || T >= ((int64_t)1 << 31))
        return MOE_ERR_UNSUPPORTED;
    // assignments, rows and blocks are counted in 32 bits
    if (T * k >= ((int64_t)1 << 31) || R >= ((int64_t)1 << 31) || T * ((H + 255) / 256) >= ((int64_t)1 << 31))
        return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if ((R > 0 && !y) || !inv_pos || !topk_w || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(inv_pos, 4) || !aligned_to(topk_w, 4)) return MOE_ERR_INVALID_ARG;
    const struct { const void* p; int64_t rows, stride; moe_dtype type; } parts[] = {
        {y, R, y_stride, dtype}, {residual, T, residual_stride, out_dtype}, {out, T, out_stride, out_dtype}};
    for (const auto& p : parts)
        if (p.p && (!aligned16(p.p) || (p.rows > 1 && (p.stride < H || p.stride * size_of(p.type) % 16))))
            return MOE_ERR_INVALID_ARG;
    Range range("moe/combine_rows");
    const CombineRowsArgs a{y, inv_pos, topk_w, residual, out, T, R, y_stride, residual_stride, out_stride, H, k};
    return finish(launch_combine_rows(dtype, out_dtype, a, (cudaStream_t)stream), nullptr, (cudaStream_t)stream);
}

}  // extern "C"
