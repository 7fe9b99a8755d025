// api_fp8.cu -- the C ABI of the 8-bit operators in include/moe.h: argument
// checks, TMA descriptors and launch sequences. Host code only.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe.h"
#include "api.h"
#include "fp8.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int32_t kNormMaxH = 32768;
static_assert(kFp8PartOffset == MOE_FP8_WORKSPACE_ZEROS, "what has to be zero lies before the parts");

moe_status check_ws(const void* ws, size_t ws_bytes, size_t need)
{
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < need) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

// The sizes of a grouped product: R rows, G weights of [N, K].
moe_status check_product(int64_t R, int32_t K, int32_t N, int32_t G, bool grouped)
{
    if (R < 0 || K <= 0 || N <= 0 || G <= 0) return MOE_ERR_INVALID_ARG;
    if (!grouped && G != 1) return MOE_ERR_INVALID_ARG;
    if (K % 16 || N % 16 || G > 256 || R >= ((int64_t)1 << 31) - 256) return MOE_ERR_UNSUPPORTED;
    // tiles are counted in 32 bits
    if ((R / 128 + G) * ((N + 127) / 128) >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

struct Operand {   // e4m3 values and their block scales
    const moe_e4m3* v;
    const float* scale;
};

Fp8GemmArgs product_args(int32_t R, int32_t K, int32_t N, int32_t G, const int32_t* offsets, const float* a_scale,
                         void* ws)
{
    unsigned char* w = static_cast<unsigned char*>(ws);
    Fp8GemmArgs a{};
    a.R = R;
    a.K = K;
    a.N = N;
    a.G = G;
    a.offsets = offsets;
    a.a_scale = a_scale;
    a.k = 1;
    a.T = R;
    a.ticket = reinterpret_cast<int32_t*>(w + kFp8TicketOffset);
    a.part = reinterpret_cast<float*>(w + kFp8PartOffset);
    a.err = reinterpret_cast<uint32_t*>(ws);
    return a;
}

// Whether a product over R rows in G groups runs two CTAs per MMA (256-row
// tiles, a third less read from L2), by rows per group on average. Measured,
// one CTA -> pair, us: gated K = 2048, N = 1408, 64 groups: 384 rows 163 -> 170,
// 768: 303 -> 284, 1536: 562 -> 516; gated K = 4096, N = 14336, 8 groups: 256:
// 266 -> 277, 512: 458 -> 448, 1024: 850 -> 793; product K = 1408, N = 2048,
// 64 groups: 768: 195 -> 207, 1536: 371 -> 365; product K = 14336, N = 4096,
// 8 groups: 1024: 391 -> 402; one group 4096 x 4096: 4096: 72 -> 71, 8192:
// 125 -> 122. Fewer rows pad more in 256-row tiles. And K is split only with one
// CTA, which pays from about 64 blocks of K on where the pairs' tiles (counted
// for equal groups) leave most of a round idle: the only round more than half, or
// the last of two or three more than 7/8. Gated, one group, K = 14336: 512 rows,
// N = 256 31 -> 48, 2048 rows, N = 256 35 -> 50, 4096 rows, N = 256 (0.42 rounds)
// 44 -> 51, 2048 rows, N = 640 (0.53) 62 -> 51, 4096 rows, N = 640 (1.05) 83 ->
// 99, 2048 rows, N = 1408, 4 groups (1.16) 137 -> 100, 8192 rows, N = 640 (2.11)
// 139 -> 151; K = 10240: 0.21 rounds 31 -> 37, 0.42 36 -> 38; K = 8192: 0.21 29 ->
// 31, 0.42 33 -> 32, 1.05 58 -> 58; K = 6144: 0.21 27 -> 25.
bool pair_for(int64_t R, int32_t K, int32_t N, int32_t G, bool gated, int sms)
{
    if (R < (int64_t)(gated ? 512 : 2048) * G) return false;
    if (K <= 64 * kFp8Block) return true;
    const int n_out = gated ? 128 : 256;
    const int64_t tiles = G * (((R + G - 1) / G + 255) / 256) * ((N + n_out - 1) / n_out);
    const int64_t pairs = sms > 1 ? sms / 2 : 1, rounds = tiles / pairs, last = tiles % pairs;
    if (rounds == 0) return 2 * last >= pairs;
    return rounds > 2 || last == 0 || 8 * last >= pairs;
}

// The form of a product: tiles of 128 columns where all of them find an SM
// (counted from above: every group may begin a tile) and the blocks are few, or
// the rows too many for a cheap join of cut tiles; else a pair as above, or one
// CTA with tiles of 256 columns. Measured, 256 / 128 columns, us, one group N =
// 4096: 8 rows K = 512 6.5 / 5.8, 4096: 11.3 / 11.9; 16 rows K = 2048 9.8 / 9.4; 64
// rows K = 4096 15.6 / 13.4; 512 rows K = 4096 19.6 / 16.0, 8192: 29.3 / 26.4,
// 12288: 36.3 / 38.0; two of 8 experts 14336 -> 4096, one row each 29.7 / 40.9; 6
// of 64 1408 -> 2048 10.5 / 11.4; 160 tiles of 128 columns on 152 SMs 20.0 / 28.0.
// A pair / 128 columns, one group N = 256: 2048 rows K = 1024 9.5 / 7.7, 8192 rows
// K = 1024 9.9 / 8.3, 4096: 19.3 / 16.9, 8192: 32.6 / 27.8; 8 groups of 2048 rows,
// N = 128, K = 2048 13.1 / 11.2.
Fp8GemmForm product_form(int64_t R, int32_t K, int32_t N, int32_t G, int sms)
{
    const int64_t m_tiles = G == 1 ? (R + 127) / 128 : R / 128 + (R < G ? R : G);
    const bool fit = m_tiles * ((N + 127) / 128) <= sms;
    if (fit && (K <= 1024 || (K <= 8192 && R >= (int64_t)16 * G))) return kFp8Narrow;
    return pair_for(R, K, N, G, false, sms) ? kFp8Pair : kFp8Wide;
}

Fp8GemmForm gated_form(int64_t R, int32_t K, int32_t F, int32_t G, int sms)
{
    return pair_for(R, K, F, G, true, sms) ? kFp8Pair : kFp8Wide;
}

moe_status run_product(Fp8GemmArgs a, const moe_e4m3* A, Operand w, bool f32, void* out, int sms, cudaStream_t s)
{
    CUtensorMap ma, mw;
    const Fp8GemmForm form = product_form(a.R, a.K, a.N, a.G, sms);
    if (!encode_map_e4m3(&ma, A, (uint64_t)a.K, (uint64_t)a.R, 0, kFp8Block, 128) ||
        !encode_map_e4m3(&mw, w.v, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.G, kFp8Block, fp8_box_rows(false, form)))
        return MOE_ERR_CUDA;
    a.w0_scale = w.scale;
    a.out = out;
    MOE_TRY(launch_fp8_gemm(f32 ? kFp8ProductF32 : kFp8ProductBf16, form, ma, mw, mw, a, sms, s));
    return MOE_OK;
}

moe_status run_gated(Fp8GemmArgs a, const moe_e4m3* A, Operand w1, Operand w3, moe_e4m3* h, float* h_scale, int sms,
                     cudaStream_t s)
{
    CUtensorMap ma, m1, m3;
    const Fp8GemmForm form = gated_form(a.R, a.K, a.N, a.G, sms);
    if (!encode_map_e4m3(&ma, A, (uint64_t)a.K, (uint64_t)a.R, 0, kFp8Block, 128) ||
        !encode_map_e4m3(&m1, w1.v, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.G, kFp8Block, fp8_box_rows(true, form)) ||
        !encode_map_e4m3(&m3, w3.v, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.G, kFp8Block, fp8_box_rows(true, form)))
        return MOE_ERR_CUDA;
    a.w0_scale = w1.scale;
    a.w1_scale = w3.scale;
    a.out = h;
    a.out_scale = h_scale;
    MOE_TRY(launch_fp8_gemm(kFp8Gated, form, ma, m1, m3, a, sms, s));
    return MOE_OK;
}

moe_status check_ffn(const moe_fp8_ffn* f)
{
    if (!f || !f->w1 || !f->w1_scale || !f->w3 || !f->w3_scale || !f->w2 || !f->w2_scale) return MOE_ERR_INVALID_ARG;
    if (!aligned16(f->w1) || !aligned16(f->w3) || !aligned16(f->w2)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// The scales behind R quantized rows of n values: 4 bytes for each block of 128
// fit into the other half of their buffer (n is a multiple of 64).
float* scales_behind(moe_e4m3* rows, size_t R, int32_t n) { return reinterpret_cast<float*>(rows + R * (size_t)n); }

// One expert set's gated product and second product; rows of the second are
// scattered to slots (src_row) or written in order to slot.
moe_status run_ffn(int32_t R, int32_t H, int32_t F, int32_t G, const int32_t* offsets, Operand x,
                   const moe_fp8_ffn& f, const int32_t* src_row, const float* topk_w, int32_t k, int64_t T, float* slot,
                   unsigned char* h, void* ws, int sms, cudaStream_t s)
{
    moe_e4m3* hq = h;
    float* hs = scales_behind(h, (size_t)R, F);
    MOE_TRY_STATUS(run_gated(product_args(R, H, F, G, offsets, x.scale, ws), x.v, {f.w1, f.w1_scale},
                             {f.w3, f.w3_scale}, hq, hs, sms, s));
    Fp8GemmArgs a = product_args(R, F, H, G, offsets, hs, ws);
    a.src_row = src_row;
    a.topk_w = topk_w;
    a.k = k;
    a.T = T;
    return run_product(a, hq, {f.w2, f.w2_scale}, /*f32=*/true, slot, sms, s);
}

// The layer's workspace: the products' part, then that of the bf16 layer, whose
// buffers for dispatched rows and h (2 bytes an element) hold the quantized rows
// and, behind them, their scales.
struct LayerLayout {
    size_t base, total;
};

LayerLayout layer_layout(const moe_dims& d)
{
    LayerLayout L;
    L.base = al256(kFp8WorkspaceBytes);
    L.total = L.base + al256(moe_workspace_size(&d));
    return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_fp8_workspace_size(const moe_dims* dims)
{
    if (!dims) return kFp8WorkspaceBytes;
    return check_dims(dims) == MOE_OK ? layer_layout(*dims).total : 0;
}

moe_status moe_add_rmsnorm_fp8(int64_t T, int32_t H, moe_dtype dtype, const void* x, int64_t x_stride,
                               const void* residual, int64_t residual_stride, const void* weight, float eps, void* sum,
                               int64_t sum_stride, void* y, moe_e4m3* q, float* scale, moe_stream_t stream)
{
    if (T < 0 || H <= 0 || !(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_BF16 && dtype != MOE_FP16 && dtype != MOE_FP32) return MOE_ERR_UNSUPPORTED;
    if (H % 16 || H > kNormMaxH || T >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    if (!x || !q || !scale) return MOE_ERR_INVALID_ARG;
    const int size = dtype == MOE_FP32 ? 4 : 2;
    const struct { const void* p; int64_t stride; } rows[] = {{x, x_stride}, {residual, residual_stride}, {sum, sum_stride}};
    for (const auto& r : rows)
        if (r.p && (!aligned16(r.p) || (T > 1 && (r.stride < H || r.stride * size % 16)))) return MOE_ERR_INVALID_ARG;
    for (const void* p : {weight, static_cast<const void*>(y), static_cast<const void*>(q)})
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    Range range("moe/add_rmsnorm_fp8");
    const Fp8NormArgs a{x, residual, weight, sum, y, q, scale, T, x_stride, residual_stride, sum_stride, H, eps};
    return finish(launch_fp8_norm(dtype, a, (cudaStream_t)stream), nullptr, (cudaStream_t)stream);
}

moe_status moe_fp8_quantize_weight(int32_t G, int32_t K, int32_t N, const moe_bf16* w, moe_e4m3* q, float* scale,
                                   moe_stream_t stream)
{
    if (G <= 0 || K <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    if (K % 16 || N % 16 || G > 256 || K > 65535 * kFp8Block) return MOE_ERR_UNSUPPORTED;
    if (!w || !q || !scale || !aligned16(w) || !aligned16(q)) return MOE_ERR_INVALID_ARG;
    Range range("moe/fp8_quantize_weight");
    return finish(launch_fp8_quantize_weight(w, q, scale, G, K, N, (cudaStream_t)stream), nullptr,
                  (cudaStream_t)stream);
}

moe_status moe_fp8_matmul(int64_t R, int32_t K, int32_t N, int32_t G, const moe_e4m3* a, const float* a_scale,
                          const int32_t* offsets, const moe_e4m3* w, const float* w_scale, moe_dtype out_dtype,
                          void* out, void* ws, size_t ws_bytes, moe_stream_t stream)
{
    MOE_TRY_STATUS(check_product(R, K, N, G, offsets != nullptr));
    if (out_dtype != MOE_BF16 && out_dtype != MOE_FP32) return MOE_ERR_UNSUPPORTED;
    MOE_TRY_STATUS(check_ws(ws, ws_bytes, kFp8WorkspaceBytes));
    if (R == 0) return MOE_OK;
    if (!a || !a_scale || !w || !w_scale || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(w) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
    const int sms = num_sms_current();
    if (sms <= 0) return MOE_ERR_CUDA;
    Range range("moe/fp8_matmul");
    MOE_TRY_STATUS(run_product(product_args((int32_t)R, K, N, G, offsets, a_scale, ws), a, {w, w_scale},
                               out_dtype == MOE_FP32, out, sms, (cudaStream_t)stream));
    return finish(cudaSuccess, ws, (cudaStream_t)stream);
}

moe_status moe_fp8_gated(int64_t R, int32_t K, int32_t F, int32_t G, const moe_e4m3* a, const float* a_scale,
                         const int32_t* offsets, const moe_e4m3* w1, const float* w1_scale, const moe_e4m3* w3,
                         const float* w3_scale, moe_e4m3* h, float* h_scale, void* ws, size_t ws_bytes,
                         moe_stream_t stream)
{
    MOE_TRY_STATUS(check_product(R, K, F, G, offsets != nullptr));
    MOE_TRY_STATUS(check_ws(ws, ws_bytes, kFp8WorkspaceBytes));
    if (R == 0) return MOE_OK;
    if (!a || !a_scale || !w1 || !w1_scale || !w3 || !w3_scale || !h || !h_scale) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(w1) || !aligned16(w3) || !aligned16(h)) return MOE_ERR_INVALID_ARG;
    const int sms = num_sms_current();
    if (sms <= 0) return MOE_ERR_CUDA;
    Range range("moe/fp8_gated");
    MOE_TRY_STATUS(run_gated(product_args((int32_t)R, K, F, G, offsets, a_scale, ws), a, {w1, w1_scale},
                             {w3, w3_scale}, h, h_scale, sms, (cudaStream_t)stream));
    return finish(cudaSuccess, ws, (cudaStream_t)stream);
}

int32_t moe_selftest_fp8_form(int64_t R, int32_t K, int32_t N, int32_t G, int32_t gated, int32_t num_sms)
{
    if (check_product(R, K, N, G, /*grouped=*/true) != MOE_OK || num_sms <= 0) return -1;
    return gated ? gated_form(R, K, N, G, num_sms) : product_form(R, K, N, G, num_sms);
}

moe_status moe_fp8_layer_forward(const moe_dims* dims, const moe_bf16* x, const moe_e4m3* xq, const float* xq_scale,
                                 const moe_bf16* Wg, const float* bias, const moe_gating* gating,
                                 const moe_fp8_ffn* routed, const moe_fp8_ffn* shared, moe_bf16* out,
                                 const moe_routing_out* routing, void* ws, size_t ws_bytes, moe_stream_t stream)
{
    MOE_TRY_STATUS(check_dims(dims));
    const moe_dims& d = *dims;
    const LayerLayout L = layer_layout(d);
    MOE_TRY_STATUS(check_ws(ws, ws_bytes, L.total));
    if (d.T == 0) return MOE_OK;
    if (!x || !xq || !xq_scale || !Wg || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(Wg) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
    MOE_TRY_STATUS(check_ffn(routed));
    if (d.F_shared > 0) MOE_TRY_STATUS(check_ffn(shared));
    const moe_bf16* shared_gate = gating ? gating->shared_gate : nullptr;
    if (shared_gate && (d.F_shared == 0 || !aligned16(shared_gate))) return MOE_ERR_INVALID_ARG;
    const int64_t R = d.T * d.k;
    MOE_TRY_STATUS(check_product(R, d.H, d.F, d.E, true));
    MOE_TRY_STATUS(check_product(R, d.F, d.H, d.E, true));
    const int sms = num_sms_current();
    if (sms <= 0) return MOE_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    unsigned char* w = static_cast<unsigned char*>(ws);
    uint32_t* err = reinterpret_cast<uint32_t*>(ws);
    const Routed rt = routed_of(d, routing, w + L.base);
    moe_plan plan;
    MOE_TRY_STATUS(moe_layer_plan(&d, &plan));

    Range layer_range("moe/fp8_layer_forward");
    Range stage("moe/route");
    MOE_TRY_STATUS(route_and_sort(d, plan.router, x, Wg, bias, gating, rt, w + L.base, err, sms, nullptr, stage, s));
    moe_e4m3* xp = rt.x_perm;
    float* xs = scales_behind(xp, (size_t)R, d.H);
    MOE_TRY(launch_fp8_dispatch(xq, xq_scale, rt.topk_idx, rt.inv_pos, rt.offsets + d.E, xp, xs, d.T, d.H, d.k, d.E, err,
                                sms, s));
    stage.next("moe/experts");
    MOE_TRY_STATUS(run_ffn((int32_t)R, d.H, d.F, d.E, rt.offsets, {xp, xs}, *routed, rt.src_row, rt.topk_w, d.k, d.T,
                           rt.slot, rt.h, ws, sms, s));
    if (d.F_shared > 0) {
        stage.next("moe/shared_expert");
        // every token, in token order, with weight 1 or the sigmoid gate's
        if (shared_gate) MOE_TRY(launch_shared_gate(x, shared_gate, rt.shared_gate, d.T, d.H, sms, s));
        MOE_TRY_STATUS(run_ffn((int32_t)d.T, d.H, d.F_shared, 1, nullptr, {xq, xq_scale}, *shared, nullptr,
                               shared_gate ? rt.shared_gate : nullptr, 1, d.T, rt.slot + (size_t)R * d.H,
                               rt.h_shared, ws, sms, s));
    }
    stage.next("moe/combine");
    MOE_TRY(launch_combine(rt.slot, d.k + (d.F_shared > 0 ? 1 : 0), out, d.T, d.H, sms, s));
    return finish(cudaSuccess, ws, s);
}

}  // extern "C"
