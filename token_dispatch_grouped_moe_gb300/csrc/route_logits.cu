// route_logits.cu -- each token's experts and weights from its logits:
//
//   s = softmax(l) or 1 / (1 + e^-l)
//   key = l without a bias (scores are in their logits' order), s + bias with one
//   a group's value = its largest key, or the sum of its two largest s (+ bias);
//     the top_groups groups of the largest values keep their experts
//   the k largest keys, ties to the lower index; w = s (/ the k's sum) * scale
//
// Which of two experts comes first is decided as in real arithmetic: in fp32
// with a bound on the keys' error, and once more in fp64 (a warp's whole row,
// `exact_row`) where two neighbours of the order are nearer than the bound. Equal
// logits with equal biases are a tie and need no second look.
//
// A warp takes a token. Its experts lie V a lane in index order, no group crossing
// a lane: lanes_per_group = the largest power of two <= 32 / groups.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.cuh"
#include "ops.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kTiny = 0x1p-96f;   // a selected score below this is looked at in fp64

// A key as an unsigned number of the same order; -0 is 0, NaN is -inf, 0 is none.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t u = __float_as_uint(v != v ? kNegInf : v + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double v)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v != v ? (double)kNegInf : v + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ float value_of(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

template <typename F> struct OrderedOf;
template <> struct OrderedOf<float> { using type = uint32_t; };
template <> struct OrderedOf<double> { using type = uint64_t; };

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// e^x within 2^-22 + 2^-23 of itself (0 below 2^-126, inf above the range): ex2's
// 2^-22, the product's rounding made good by its residual
__device__ __forceinline__ float exp_near(float x)
{
    constexpr float kLog2e = 1.44269504088896340736f;
    constexpr float kLog2eLow = 1.925963033500e-8f;   // log2(e) - kLog2e
    constexpr float kLn2 = 0.69314718055994530942f;
    x = fminf(fmaxf(x, -120.0f), 120.0f);
    const float n = x * kLog2e;
    const float r = fmaf(x, kLog2e, -n) + x * kLog2eLow;
    return ex2(n) * fmaf(r, kLn2, 1.0f);
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

// Where a lane's experts lie.
template <int V>
struct Place {
    int group, first, n;   // its group, its first expert, how many it has (0: none)
    int lanes;             // lanes of a group

    __device__ __forceinline__ Place(const RouteLogitsArgs& a, int lane)
    {
        lanes = 32 / a.groups;
        lanes = 1 << (31 - __clz(lanes));
        const int size = a.E / a.groups;
        group = lane / lanes;
        const int at = (lane % lanes) * V;
        first = group * size + at;
        n = group < a.groups ? max(0, min(V, size - at)) : 0;
    }
};

template <int V, typename T>
__device__ __forceinline__ void load_row(const RouteLogitsArgs& a, int64_t t, const Place<V>& p, float (&l)[V])
{
    const T* row = static_cast<const T*>(a.logits) + t * a.stride + p.first;
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = j < p.n ? to_float(row[j]) : kNegInf;
}

template <int V>
__device__ __forceinline__ void load_bias(const RouteLogitsArgs& a, const Place<V>& p, float (&b)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = a.bias && j < p.n ? __ldg(a.bias + p.first + j) : 0.0f;
}

template <int V>
__device__ __forceinline__ float row_max(const float (&l)[V])
{
    float m = l[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
    return value_of(warp_max(ordered(m)));
}

// The order of a row from its scores: lane r < k gets the r-th expert, its score
// and its logit. near (fp32 only): whether neighbours that the order depends on
// are within 2 tol of one another (the sums of two: 8 tol), tol bounding the error
// of s + bias.
template <int V, typename F>
__device__ __forceinline__ bool order_row(const RouteLogitsArgs& a, const Place<V>& p, int lane, const float (&l)[V],
                                          const float (&b)[V], const F (&s)[V], F tol, int& id, F& score, float& logit)
{
    using U = typename OrderedOf<F>::type;
    constexpr bool CHECK = sizeof(F) == 4;
    const bool biased = a.bias != nullptr;
    bool near = false;
    U key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = j < p.n ? ordered(biased ? s[j] + (F)b[j] : (F)l[j]) : (U)0;
    if (a.groups > 1) {
        U value;
        if (a.group_top == 1) {
            value = key[0];
#pragma unroll
            for (int j = 1; j < V; ++j) value = max(value, key[j]);
            for (int d = 1; d < p.lanes; d <<= 1) value = max(value, __shfl_xor_sync(kAll, value, d));
        } else {
            // the two largest of the lane, then of the group
            F x = -__builtin_huge_val(), y = x;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                F c = s[j] + (F)b[j];
                if (j >= p.n || c != c) c = -__builtin_huge_val();
                y = max(y, min(x, c));
                x = max(x, c);
            }
            for (int d = 1; d < p.lanes; d <<= 1) {
                const F ox = __shfl_xor_sync(kAll, x, d), oy = __shfl_xor_sync(kAll, y, d);
                y = max(max(y, oy), min(x, ox));
                x = max(x, ox);
            }
            value = ordered(x + y);   // -inf + inf: counts as -inf
        }
        int place = 0;
        U kept_least = ~(U)0, left_most = 0;
        for (int g = 0; g < a.groups; ++g) {
            const U v = __shfl_sync(kAll, value, g * p.lanes);
            place += v > value || (v == value && g < p.group);
        }
        const bool kept = place < a.top_groups;
        if constexpr (CHECK) {
            if (biased || a.group_top == 2) {
                kept_least = kept && p.group < a.groups ? value : ~(U)0;
                left_most = kept || p.group >= a.groups ? 0 : value;
                kept_least = __reduce_min_sync(kAll, kept_least);
                left_most = __reduce_max_sync(kAll, left_most);
                if (left_most) {
                    const float x = value_of(kept_least), y = value_of(left_most);
                    near = !(x - y > (a.group_top == 1 ? 2.0f : 8.0f) * tol) && !(x == kNegInf && y == kNegInf);
                }
            }
        }
        if (!kept) {
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = 0;
        }
    }
    U best = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) best = max(best, key[j]);
    U before = 0;
    float l_before = 0.0f, b_before = 0.0f;
    for (int r = 0; r < a.k; ++r) {
        const U top = warp_max(best);
        const int from = __ffs((int)__ballot_sync(kAll, best == top)) - 1;
        int jw = 0;
        float lw = 0.0f, bw = 0.0f;
        F sw = 0;
#pragma unroll
        for (int j = V - 1; j >= 0; --j)
            if (key[j] == top) { jw = j; lw = l[j]; bw = b[j]; sw = s[j]; }
        if (lane == from) {
            best = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (j == jw) key[j] = 0;
                best = max(best, key[j]);
            }
        }
        const int e = __shfl_sync(kAll, p.first + jw, from);
        sw = __shfl_sync(kAll, sw, from);
        lw = __shfl_sync(kAll, lw, from);
        if constexpr (CHECK) {
            if (biased) {
                bw = __shfl_sync(kAll, bw, from);
                if (r > 0) {
                    const float x = value_of(before), y = value_of(top);
                    const bool tie = (lw == l_before && bw == b_before) || (x == kNegInf && y == kNegInf);
                    near = near || (!tie && !(x - y > 2.0f * tol));
                }
                before = top;
                l_before = lw;
                b_before = bw;
            }
        }
        if (lane == r) { id = e; score = sw; logit = lw; }
    }
    if constexpr (CHECK) {
        // any expert left that is near the last one selected and not its equal
        if (biased) {
            const float x = value_of(before);
            bool left = false;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float y = value_of(key[j]);
                const bool tie = (l[j] == l_before && b[j] == b_before) || (x == kNegInf && y == kNegInf);
                left = left || (key[j] != 0 && !tie && !(x - y > 2.0f * tol));
            }
            near = near || __any_sync(kAll, left);
        }
    }
    return near;
}

__device__ __forceinline__ void store_row(const RouteLogitsArgs& a, int64_t t, int lane, int id, float w)
{
    if (lane < a.k) {
        a.topk_idx[t * a.k + lane] = id;
        a.topk_w[t * a.k + lane] = w;
    }
}

// A row in fp64: where fp32 does not tell two experts apart, and rows with a NaN
// or an infinite score.
template <int V, typename T>
__device__ __noinline__ void exact_row(const RouteLogitsArgs& a, int64_t t, int lane)
{
    const Place<V> p(a, lane);
    float l[V], b[V];
    double s[V];
    load_row<V, T>(a, t, p, l);
    load_bias<V>(a, p, b);
    bool nan = false;
#pragma unroll
    for (int j = 0; j < V; ++j) nan = nan || l[j] != l[j];
    nan = __any_sync(kAll, nan);
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 1.0 / (1.0 + exp(-(double)l[j]));
    } else {
        double m = row_max<V>(l);
        if (m == (double)kNegInf) m = 0.0;   // a row of nothing: scores 0
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s[j] = exp((double)l[j] - m);
            if (j < p.n) sum += s[j];
        }
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = sum == 0.0 ? 0.0 : s[j] / sum;
    }
    int id = 0;
    double score = 0.0;
    float logit = 0.0f;
    order_row<V, double>(a, p, lane, l, b, s, 0.0, id, score, logit);
    double w = lane < a.k ? score : 0.0;
    if (a.renorm) {
        double sum = w;
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        w = sum == 0.0 ? 0.0 : w / sum;
    }
    w *= (double)a.scale;
    store_row(a, t, lane, id, nan ? __int_as_float(0x7fc00000) : (float)w);
}

template <int V, typename T>
__global__ void __launch_bounds__(32 * kWarps) route_logits_kernel(const RouteLogitsArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const Place<V> p(a, lane);
    float b[V];
    load_bias<V>(a, p, b);
    float b_most = 0.0f;   // the largest finite |bias|
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (fabsf(b[j]) < __builtin_huge_valf()) b_most = fmaxf(b_most, fabsf(b[j]));
    b_most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(b_most)));

    for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += (int64_t)gridDim.x * kWarps) {
        float l[V], s[V];
        load_row<V, T>(a, t, p, l);
        bool bad = false;
#pragma unroll
        for (int j = 0; j < V; ++j) bad = bad || !(l[j] < __builtin_huge_valf());
        float s_most, tol;
        if (a.sigmoid) {
            // 1 + e and the reciprocal: within 2.25 * 2^-22 of the score
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = rcp(1.0f + exp_near(-l[j]));
            s_most = 1.0f;
            tol = 2.5f * 0x1p-22f;
        } else {
            // e^d within (|d| / 2 + 3) 2^-23 of itself (d's own rounding), the sum of
            // up to 256 (lane by lane, then 5 steps) within 17 * 2^-23: together less
            // than 24 * 2^-23 of the largest score, for every expert
            float m = row_max<V>(l);
            if (m == kNegInf) m = 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[j] = exp_near(l[j] - m);
                sum += s[j];
            }
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
            const float inv = sum > 0.0f ? rcp(sum) : 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] *= inv;
            s_most = inv;
            tol = 24.0f * 0x1p-23f * inv;
        }
        tol += 0x1p-24f * (s_most + b_most) + 0x1p-90f;
        int id = 0;
        float score = 0.0f, logit = 0.0f;
        bool again = order_row<V, float>(a, p, lane, l, b, s, tol, id, score, logit) || __any_sync(kAll, bad);
        float w = lane < a.k ? score : 0.0f;
        if (a.renorm) {
            again = again || __any_sync(kAll, lane < a.k && score < kTiny && logit > kNegInf);
            float sum = w;
            for (int d = 4; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
            w = sum > 0.0f ? __fdividef(w, sum) : 0.0f;
        }
        if (again) exact_row<V, T>(a, t, lane);
        else store_row(a, t, lane, id, w * a.scale);
    }
}

template <int V, typename T>
cudaError_t launch(const RouteLogitsArgs& a, int num_sms, cudaStream_t s)
{
    int64_t blocks = (a.T + kWarps - 1) / kWarps;
    const int64_t most = (int64_t)num_sms * 8;
    if (blocks > most) blocks = most;
    return launch_pdl(route_logits_kernel<V, T>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, s, a);
}

template <typename T>
cudaError_t launch_type(const RouteLogitsArgs& a, int num_sms, cudaStream_t s)
{
    int lanes = 32 / a.groups;
    while (lanes & (lanes - 1)) lanes &= lanes - 1;
    const int per_lane = (a.E / a.groups + lanes - 1) / lanes;
    if (per_lane <= 1) return launch<1, T>(a, num_sms, s);
    if (per_lane <= 2) return launch<2, T>(a, num_sms, s);
    if (per_lane <= 4) return launch<4, T>(a, num_sms, s);
    if (per_lane <= 8) return launch<8, T>(a, num_sms, s);
    if (per_lane <= 16) return launch<16, T>(a, num_sms, s);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_route_logits(moe_dtype dtype, const RouteLogitsArgs& a, int num_sms, cudaStream_t s)
{
    if (a.T == 0) return cudaSuccess;
    switch (dtype) {
    case MOE_BF16: return launch_type<__nv_bfloat16>(a, num_sms, s);
    case MOE_FP16: return launch_type<__half>(a, num_sms, s);
    case MOE_FP32: return launch_type<float>(a, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
