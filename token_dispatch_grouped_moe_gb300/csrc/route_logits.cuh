// route_logits.cuh -- each token's experts and weights from its logits:
//
//   s = softmax(l) or 1 / (1 + e^-l)
//   key = l without a bias (scores are in their logits' order), s + bias with one
//   a group's value = its largest key, or the sum of its two largest s (+ bias);
//     the top_groups groups of the largest values keep their experts
//   the k largest keys, ties to the lower index; w = s (/ the k's sum) * scale
//
// Which of two experts comes first is decided as in real arithmetic: in fp32
// with a bound on the keys' error, and in fp64 where two neighbours of the order are
// nearer than the bound. Equal logits with equal biases are a tie, by index.
//
// A warp takes a token, its experts V a lane in index order, no group crossing a lane
// (lanes_per_group = the largest power of two <= 32 / groups). Its scores are computed
// once, approximately; the groups' values and then the lanes' best are passed from the
// top down with the warp's maximum until enough are passed; the ten or so experts that
// are left go one to a lane, two tokens to a warp, and are ranked there by comparing each
// with each. So nothing is sorted, and no step looks at all experts more than once.
//
// What bounds it (one GB300): its instructions, 330 a token (8 of 256 by their logits),
// 620 with scores, bias and groups, at two thirds of the issue rate, and not the memory:
// 32768 tokens x 256 fp32 logits, top 8, us: by logits 15.2, sigmoid with bias 20, and
// with 4 of 8 groups by the sum of their two best 26 (the logits' bytes: 5); top 2 of 8
// 7.8; 5003 x 160 in 8 groups 7.0; one token 2.3, as any launch. One row in a thousand
// wants fp64, 1.5 us of its warp's time; a softmax with a bias, where its sum has to be
// taken again, 9 (28 us without groups, 32 with: the last such row ends the launch).
// 15 local accesses a token by logits, 44 with scores, bias and groups, are in it at 48
// registers; they are not the limit's alone: compiled for 64 and 80 (4 and 3 blocks an SM
// instead of 5) a thread still spills 41 and 42 registers and loads 97 and 98 in place of 62
// and 135, and the third of the times above is 26.7 and 31 us.
// Measured on the way, the third of these (us): each of the k maxima by a search of all
// registers 122; fp64 in functions that were unrolled, cold code fetched for 40 us, 62; in
// calls from the loop, which spill its registers, 29.
#pragma once

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
__device__ __forceinline__ double value64(uint64_t u)
{
    return __longlong_as_double((long long)(u >> 63 ? u ^ (1ull << 63) : ~u));
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

// The warp's largest value (a NaN gives way).
__device__ __forceinline__ float max_f32(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float max_or_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float kLog2e = 1.44269504088896340736f;

// e^x within 2^-22 + 2^-23 of itself (0 below 2^-126, inf above the range): ex2's
// 2^-22, the product's rounding made good by its residual
__device__ __forceinline__ float exp_near(float x)
{
    constexpr float kLog2eLow = 1.925963033500e-8f;   // log2(e) - kLog2e
    constexpr float kLn2 = 0.69314718055994530942f;
    x = fminf(fmaxf(x, -120.0f), 120.0f);
    const float n = x * kLog2e;
    const float r = fmaf(x, kLog2e, -n) + x * kLog2eLow;
    return ex2(n) * fmaf(r, kLn2, 1.0f);
}

__device__ __forceinline__ float sigmoid_near(float x) { return rcp(1.0f + exp_near(-x)); }

// How far a key in fp32 may be from itself, beside what all keys of its row share.
// Sigmoid: s (1 - s) times e^-x's error (2^-22, and of a plain product with log2(e) 2 |x|
// 2^-24, where |x| s (1 - s) < 1/4), a sum and a reciprocal: 4.5 * 2^-24; softmax, in the
// largest score (`most` = 1 / the sum): e^d within (6 + 3 |d|) 2^-24 of itself, times e^d
// less than 7 * 2^-24; and the key's own rounding. A softmax's sum of up to 256 (within
// (22.5 + 21) 2^-24: 16 in a lane, 5 steps), its reciprocal and the product scale all
// scores of a row alike, by 47 * 2^-24 at most. That moves two scores against one another
// by as much of their difference, and keys as near as this matters for have scores as
// different as their biases, 2 b_most at most.
__device__ __forceinline__ float sigmoid_tol(float b_most) { return 5.0f * 0x1p-24f + 0x1p-24f * (1.0f + b_most); }
__device__ __forceinline__ float softmax_tol(float most, float b_most)
{
    return 7.0f * 0x1p-24f * most + 24.0f * 0x1p-24f * fminf(2.0f * b_most, most) + 0x1p-24f * (most + b_most);
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

template <typename T>
__device__ __forceinline__ const T* row_of(const RouteLogitsArgs& a, int64_t t)
{
    return static_cast<const T*>(a.logits) + t * a.stride;
}

template <int V, typename T>
__device__ __forceinline__ void load_row(const T* row, const Place<V>& p, float (&l)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) l[j] = j < p.n ? to_float(row[p.first + j]) : kNegInf;
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
    load_row<V, T>(row_of<T>(a, t), p, l);
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

// A row with every expert's key kept, in fp32 with the bounds above, and in fp64
// where they do not decide: rows that the short way below does not take.
template <int V, typename T>
__device__ __noinline__ void careful_row(const RouteLogitsArgs& a, int64_t t, int lane, float b_most)
{
    const Place<V> p(a, lane);
    float l[V], b[V], s[V];
    load_row<V, T>(row_of<T>(a, t), p, l);
    load_bias<V>(a, p, b);
    bool bad = false;
#pragma unroll
    for (int j = 0; j < V; ++j) bad = bad || !(l[j] < __builtin_huge_valf());
    float tol;
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = sigmoid_near(l[j]);
        tol = sigmoid_tol(b_most);
    } else {
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
        tol = softmax_tol(inv, b_most);
    }
    tol += 0x1p-90f;
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

// 16 bytes, or all of them, of a lane's logits at a time
template <int V, typename T>
__device__ __forceinline__ void load_whole(const T* p, float (&l)[V])
{
    constexpr int BYTES = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;
    constexpr int N = BYTES / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < V; j += N) {
        alignas(16) T v[N];
        if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(v) = __ldg(reinterpret_cast<const uint4*>(p + j));
        else if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(v) = __ldg(reinterpret_cast<const uint2*>(p + j));
        else if constexpr (BYTES == 4) *reinterpret_cast<uint32_t*>(v) = __ldg(reinterpret_cast<const uint32_t*>(p + j));
        else v[0] = p[j];
#pragma unroll
        for (int i = 0; i < N; ++i) l[j + i] = to_float(v[i]);
    }
}

// The two largest of two pairs, each ordered.
__device__ __forceinline__ void merge_two(float& x, float& y, float ox, float oy)
{
    const float lo = fminf(x, ox);
    x = fmaxf(x, ox);
    y = fmaxf(fmaxf(y, oy), lo);
}

// e^x in fp64, |x| up to 700 (beyond: of 700): 2^n e^r, |r| <= ln(2) / 2, by the power
// series of e^r up to r^13. (What follows in fp64 is inlined, without calls: with calls from
// the short way's loop, for which its registers are spilled, 29 us instead of 26.)
__device__ __forceinline__ double exp64(double x)
{
    constexpr double kLog2e64 = 1.4426950408889634074, kLn2High = 0.69314718055994530942, kLn2Low = 2.3190468138462996e-17;
    x = fmin(fmax(x, -700.0), 700.0);
    const double n = rint(x * kLog2e64);
    const double r = fma(-n, kLn2Low, fma(-n, kLn2High, x));
    double p = 1.0 / 6227020800.0;   // 1 / 13!
    constexpr double kInverse[13] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0,
                                     1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0};
#pragma unroll
    for (int i = 0; i < 13; ++i) p = fma(p, r, kInverse[i]);
    return p * __longlong_as_double((long long)((int)n + 1023) << 52);
}

// 1 / d for 1 <= d <= 256: rcp's 22 bits, doubled twice by Newton's iteration.
__device__ __forceinline__ double inverse64(double d)
{
    double y = (double)rcp((float)d);
    y = fma(y, fma(-d, y, 1.0), y);
    return fma(y, fma(-d, y, 1.0), y);
}

// A score in fp64; softmax: from the largest logit and 1 / the sum.
__device__ __forceinline__ double score64(float l, int sigmoid, float m, double inv)
{
    if (!sigmoid) return exp64((double)l - (double)m) * inv;
    const double t = exp64(-fabs((double)l));
    return (l < 0.0f ? t : 1.0) * inverse64(1.0 + t);
}

// 1 / the sum of e^(l - m) over a row in fp64 (four at a time: it is cold, and short).
template <typename T>
__device__ __forceinline__ double inverse_sum64(const T* row, int first, int n, float m)
{
    double sum = 0.0;
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += 4) {
        double v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = exp64((double)to_float(row[first + min(j0 + i, n - 1)]) - (double)m);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += j0 + i < n ? v[i] : 0.0;
    }
#pragma unroll 1
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    return inverse64(sum);
}

// Which groups are kept, by values in fp64: lane i < total has the score + bias
// `key` of an expert of `group`, the lanes together all that may be among a group's
// one (or two) largest. A bit a group.
__device__ __forceinline__ unsigned settle_groups(const RouteLogitsArgs& a, int lane, int total, int group, double key)
{
    const uint64_t mine = ordered(key);   // (compared as whole numbers: fp64 is slow)
    uint64_t x = 0, y = 0;                // lane g: the two largest of group g
    for (int i = 0; i < total; ++i) {
        const uint64_t k = __shfl_sync(kAll, mine, i);
        const int g = __shfl_sync(kAll, group, i);
        if (g != lane) continue;
        if (k > x) { y = x; x = k; }
        else if (k > y) y = k;
    }
    const uint64_t value = a.group_top == 2 ? ordered(value64(x) + value64(y)) : x;
    int place = 0;
    for (int g = 0; g < a.groups; ++g) {
        const uint64_t v = __shfl_sync(kAll, value, g);
        place += v > value || (v == value && g < lane);
    }
    return __ballot_sync(kAll, lane < a.groups && place < a.top_groups);
}

// Lists the experts of the lanes with `mine` whose v is at least `least` in `list`, in
// index order; how many there are (over 32: none is listed).
template <int V>
__device__ __forceinline__ int list_experts(uint8_t* list, int lane, const float (&v)[V], int first, int n, bool mine,
                                            float least)
{
    unsigned bits = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (v[j] >= least && j < n) bits |= 1u << j;
    if (!mine) bits = 0;
    const int count = __popc(bits);
    int at = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, at, d);
        if (lane >= d) at += o;
    }
    const int total = __shfl_sync(kAll, at, 31);
    if (total > 32) return total;
    uint8_t* to = list + at - count;
    __syncwarp();
    for (; bits; bits &= bits - 1) *to++ = (uint8_t)(first + __ffs((int)bits) - 1);   // one or two
    __syncwarp();
    return total;
}

// What the keys are: the logits (scores are in their order; group values too), or
// scores + bias, or the logits with group values that are sums of two scores.
enum RouteKeys { kByLogit = 0, kByBiased = 1, kByPairs = 2 };

// A row after its scan: the experts among which its k are, and what their scores and
// order are computed with.
struct Scanned {
    int total;            // listed; over 32: the row takes a longer way
    float m, inv, tol;    // softmax: the largest logit, 1 / the sum; the bound on a key's error
};

// The scores, the groups, then a bound that at least k keys reach: the k-th largest of
// the lanes' best. The few experts that reach it are listed.
template <int V, typename T, bool FULL, RouteKeys KEYS>
__device__ __forceinline__ Scanned scan_row(const RouteLogitsArgs& a, const Place<V>& p, int n, int lane, const T* row,
                                            const float (&l)[V], const float (&b)[V], float b_most, uint8_t* list)
{
    Scanned r{33, 0.0f, 1.0f, 0.0f};
    float c[V];   // scores + bias
    if (!a.sigmoid && (KEYS != kByLogit || !a.renorm)) {
        float m = l[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = fmaxf(m, l[j]);
        r.m = max_f32(FULL || n > 0 ? m : kNegInf);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            c[j] = ex2((l[j] - r.m) * kLog2e);
            if (FULL || j < n) sum += c[j];
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        r.inv = rcp(sum);   // a row of -inf, or with +inf or NaN: NaN
        if (!(sum < __builtin_huge_valf())) return r;
        if constexpr (KEYS != kByLogit) {
#pragma unroll
            for (int j = 0; j < V; ++j) c[j] = KEYS == kByBiased ? fmaf(c[j], r.inv, b[j]) : c[j] * r.inv;
            r.tol = softmax_tol(r.inv, b_most);
        }
    } else if constexpr (KEYS != kByLogit) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            c[j] = rcp(1.0f + ex2(-kLog2e * l[j]));
            if (KEYS == kByBiased) c[j] += b[j];
        }
        r.tol = sigmoid_tol(b_most);
    }
    float key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = FULL || j < n ? (KEYS == kByBiased ? c[j] : l[j]) : kNegInf;
    float best = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) best = max_or_nan(best, key[j]);
    // a NaN logit or bias; +inf as a logit
    if (__any_sync(kAll, KEYS == kByBiased ? best != best : !(best < __builtin_huge_valf()))) return r;
    bool kept = FULL || n > 0;
    if (a.groups > 1) {
        float value, last;   // of the group; the least of what makes it up
        if constexpr (KEYS == kByBiased || KEYS == kByPairs) {
            if (a.group_top == 2) {
                constexpr int H = V > 1 ? V / 2 : 1;
                float x[H], y[H];
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    const float u = FULL || 2 * j < n ? c[2 * j] : kNegInf;
                    const float v = V > 1 && (FULL || 2 * j + 1 < n) ? c[V > 1 ? 2 * j + 1 : 0] : kNegInf;
                    x[j] = fmaxf(u, v);
                    y[j] = fminf(u, v);
                }
#pragma unroll
                for (int w = 1; w < H; w <<= 1)
#pragma unroll
                    for (int j = 0; j < H; j += 2 * w) merge_two(x[j], y[j], x[j + w], y[j + w]);
                for (int d = 1; d < p.lanes; d <<= 1)
                    merge_two(x[0], y[0], __shfl_xor_sync(kAll, x[0], d), __shfl_xor_sync(kAll, y[0], d));
                value = x[0] + y[0];
                last = y[0];
            }
        }
        if (KEYS == kByLogit || a.group_top != 2) {
            value = best;
            for (int d = 1; d < p.lanes; d <<= 1) value = fmaxf(value, __shfl_xor_sync(kAll, value, d));
            last = value;
        }
        // down the groups' values until enough groups have been passed
        const bool leads = (lane & (p.lanes - 1)) == 0 && (FULL || n > 0);
        float rest = value, least;
        unsigned equal;   // the groups of the last value, by their first lanes
        int have = 0;
        for (;;) {
            least = max_f32(rest);
            if (!(least > kNegInf)) return r;
            equal = __ballot_sync(kAll, leads && rest == least);
            have += __popc(equal);
            if (have >= a.top_groups) break;
            if (rest == least) rest = kNegInf;
        }
        bool near = false;
        if constexpr (KEYS != kByLogit) {
            // equal values across the border, or the next one not well below
            const float next = max_f32(value < least ? value : kNegInf);
            near = have > a.top_groups || !(least - next > (a.group_top == 2 ? 8.0f : 2.0f) * r.tol);
        }
        // of the groups of the last value those of the lowest index
        const unsigned lower = equal & ((1u << (p.group * p.lanes)) - 1u);
        kept = kept && (value > least || (value == least && __popc(lower) < a.top_groups - have + __popc(equal)));
        if (KEYS != kByLogit && near) {
            const float(&from)[V] = KEYS == kByPairs ? c : key;
            const int total = list_experts<V>(list, lane, from, p.first, n, FULL || n > 0, last - 2.0f * r.tol);
            if (total > 32) return r;
            const int e = lane < total ? list[lane] : 0;
            const float le = to_float(row[e]);
            // (without a bias the sum does not matter)
            const double inv = KEYS == kByPairs || a.sigmoid ? (double)r.inv : inverse_sum64<T>(row, p.first, n, r.m);
            const double k64 = score64(le, a.sigmoid, r.m, inv) + (KEYS == kByBiased ? (double)__ldg(a.bias + e) : 0.0);
            const unsigned mask = settle_groups(a, lane, total, e / (a.E / a.groups), k64);
            kept = n > 0 && ((mask >> p.group) & 1u);
        }
        if (!kept) best = kNegInf;
    }
    if constexpr (V == 1) {
        if (a.groups == 1 && a.E <= 16) {   // all of them (32768 tokens, top 2 of 8: 11.1 -> 9.9 us)
            if (lane < a.E) list[lane] = (uint8_t)lane;
            __syncwarp();
            r.total = a.E;
            return r;
        }
    }
    // at least k keys (or all) are as large as the k-th largest of the lanes' best
    float least = kNegInf;
    for (int i = 0; i < a.k; ++i) {
        least = max_f32(best);
        if (best == least) best = kNegInf;
    }
    r.total = list_experts<V>(list, lane, key, p.first, n, kept, least - 2.0f * r.tol);
    return r;
}

// The rows (a bit each) of the halves of a warp (W = 16), or its one row, that have a
// lane with `which`.
template <int W>
__device__ __forceinline__ unsigned rows_with(bool which)
{
    const unsigned lanes = __ballot_sync(kAll, which);
    return W == 16 ? (unsigned)((lanes & 0xffffu) != 0) | (unsigned)((lanes >> 16) != 0) << 1 : (unsigned)(lanes != 0);
}

// The listed experts of a row, one to each of W lanes (32, or 16 and another row in the
// other half of the warp): their order, in fp64
// where fp32 does not tell it, and the k weights. Returns the rows (a bit each)
// that are not stored: whose scores are too small for fp32.
template <int V, typename T, RouteKeys KEYS, int W>
__device__ __forceinline__ unsigned order_listed(const RouteLogitsArgs& a, const Place<V>& p, int n, int lane, int64_t t0,
                                                 const uint8_t* list, const Scanned& r0, const Scanned& r1)
{
    const bool second = W == 16 && lane >= 16;
    const int sub = lane & (W - 1);
    const int64_t t = t0 + second;
    const T* row = row_of<T>(a, t);
    const int total = second ? r1.total : r0.total;
    const float m = second ? r1.m : r0.m, inv = second ? r1.inv : r0.inv, tol = second ? r1.tol : r0.tol;
    const int most = W == 16 ? max(r0.total, r1.total) : r0.total;
    const bool mine = sub < total;
    const int e = mine ? list[(second ? 32 : 0) + sub] : 0;
    const float le = mine ? to_float(row[e]) : kNegInf;
    int place = 0;
    float s;
    unsigned later = 0;
    if constexpr (KEYS == kByBiased) {
        const float be = __ldg(a.bias + e);
        s = a.sigmoid ? sigmoid_near(le) : exp_near(le - m) * inv;
        // before this one for certain, and before it or equal to it as far as fp32 tells
        const float k = mine ? s + be : kNegInf, far = k + 2.0f * tol, close = k - 2.0f * tol;
        int maybe = 0;
        for (int i = 0; i < most; i += 4) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // (lanes behind the last listed: -inf)
                const float o = __shfl_sync(kAll, k, i + q, W);
                if (o > far) ++place;
                if (o >= close) ++maybe;
            }
        }
        bool open = __any_sync(kAll, mine && place < a.k && maybe - place != 1);
        if (open && !a.sigmoid) {
            // fp64 but for the sum over all experts, whose error moves two keys against one
            // another by 47 * 2^-24 of their scores' difference; compared as pairs of fp32
            const double s64 = score64(le, 0, m, (double)inv), k64 = s64 + (double)be;
            // (an infinite key, of an infinite bias, has no low part and no error: equal ones are a tie)
            const float high = mine ? (float)k64 : kNegInf, s32 = (float)s64;
            const float size = fabsf(high) < __builtin_huge_valf() ? fabsf(high) : 0.0f;
            const float low = fabsf(high) < __builtin_huge_valf() ? (float)(k64 - (double)high) : 0.0f;
            place = maybe = 0;
#pragma unroll 4
            for (int i = 0; i < most; ++i) {
                const float oh = __shfl_sync(kAll, high, i, W), ol = __shfl_sync(kAll, low, i, W);
                const float os = __shfl_sync(kAll, s32, i, W);
                const float d = (oh - high) + (ol - low), u = 48.0f * 0x1p-24f * fabsf(os - s32) + 0x1p-44f * size;
                const bool same = oh == high && ol == low && (os == s32 || !(fabsf(oh) < __builtin_huge_valf()));
                const bool first = same ? i < sub : d > u;
                place += first;
                maybe += first || (!same && d >= -u);
            }
            open = __any_sync(kAll, mine && place < a.k && maybe != place);
        }
        if (open) {
            // ties by index
            double inv64 = 1.0;
            if (!a.sigmoid) {
                inv64 = inverse_sum64<T>(row_of<T>(a, t0), p.first, n, r0.m);
                if (W == 16 && r1.total) {
                    const double other = inverse_sum64<T>(row_of<T>(a, t0 + 1), p.first, n, r1.m);
                    if (second) inv64 = other;
                }
            }
            // (compared as whole numbers: fp64 is slow)
            const uint64_t k64 = mine ? ordered(score64(le, a.sigmoid, m, inv64) + (double)be) : 0;
            place = 0;
#pragma unroll 4
            for (int i = 0; i < most; ++i) {
                const uint64_t o = __shfl_sync(kAll, k64, i, W);
                place += o > k64 || (o == k64 && i < sub);
            }
        }
    } else {
        for (int i = 0; i < most; i += 4) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float o = __shfl_sync(kAll, le, i + q, W);
                if (o > le || (o == le && i + q < sub)) ++place;
            }
        }
        float from = m;
        if (KEYS == kByLogit && !a.sigmoid && a.renorm) {
            // the sum over all experts cancels
            from = le;
#pragma unroll
            for (int d = W / 2; d > 0; d >>= 1) from = fmaxf(from, __shfl_xor_sync(kAll, from, d));
        }
        s = a.sigmoid ? sigmoid_near(le) : exp_near(le - from) * inv;
    }
    const bool chosen = mine && place < a.k;
    if (a.renorm) {
        later |= rows_with<W>(chosen && s < kTiny);
        float sum = chosen ? s : 0.0f;
#pragma unroll
        for (int d = W / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        s = __fdividef(s, sum);
    }
    if (chosen && !((later >> second) & 1u)) {
        a.topk_idx[t * a.k + place] = e;
        a.topk_w[t * a.k + place] = s * a.scale;
    }
    return later;
}

// The short way, which nearly every row takes: two rows a warp are scanned, then their
// listed experts put in order side by side. FULL: every lane holds V experts, and they
// may be read in vectors.
template <int V, typename T, bool FULL, RouteKeys KEYS>
__global__ void __launch_bounds__(32 * kWarps, V <= 8 ? 5 : 2) route_logits_kernel(const __grid_constant__ RouteLogitsArgs a)
{
    __shared__ uint8_t listed[kWarps][64];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    uint8_t* list = listed[threadIdx.x >> 5];
    const Place<V> p(a, lane);
    const int n = FULL ? V : p.n;
    float b[V];
    float b_most = 0.0f;   // the largest finite |bias|
    if constexpr (KEYS == kByBiased) {
        load_bias<V>(a, p, b);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (fabsf(b[j]) < __builtin_huge_valf()) b_most = fmaxf(b_most, fabsf(b[j]));
        b_most = max_f32(b_most);
    }
    const int per = a.rows_per_warp;
    for (int64_t t = per * ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)); t < a.T; t += per * (int64_t)gridDim.x * kWarps) {
        const bool two = per == 2 && t + 1 < a.T;
        const T *row0 = row_of<T>(a, t), *row1 = row_of<T>(a, two ? t + 1 : t);
        float l0[V], l1[V];
        if constexpr (FULL) {
            load_whole<V, T>(row0 + p.first, l0);
            load_whole<V, T>(row1 + p.first, l1);
        } else {
            load_row<V, T>(row0, p, l0);
            load_row<V, T>(row1, p, l1);
        }
        const Scanned r0 = scan_row<V, T, FULL, KEYS>(a, p, n, lane, row0, l0, b, b_most, list);
        Scanned r1{0, 0.0f, 1.0f, 0.0f};
        if (two) r1 = scan_row<V, T, FULL, KEYS>(a, p, n, lane, row1, l1, b, b_most, list + 32);
        unsigned later = 0;   // of the two rows
        if (r0.total <= 16 && r1.total <= 16) {
            later = order_listed<V, T, KEYS, 16>(a, p, n, lane, t, list, r0, r1);
        } else {
            later = 1;
            if (r0.total <= 32) later = order_listed<V, T, KEYS, 32>(a, p, n, lane, t, list, r0, r0);
            if (r1.total > 32) later |= 2;
            else if (r1.total) later |= order_listed<V, T, KEYS, 32>(a, p, n, lane, t + 1, list + 32, r1, r1) << 1;
        }
        __syncwarp();
        for (; later; later &= later - 1) careful_row<16, T>(a, t + (later & 1u ? 0 : 1), lane, b_most);
    }
}

template <int V, typename T, bool FULL, RouteKeys KEYS>
cudaError_t launch(RouteLogitsArgs a, int num_sms, cudaStream_t s)
{
    // two rows a warp, or one where there are not more rows than warps at a time
    const int64_t most = (int64_t)num_sms * 8;
    a.rows_per_warp = a.T <= (int64_t)num_sms * 5 * kWarps ? 1 : 2;
    int64_t blocks = (a.T + a.rows_per_warp * kWarps - 1) / (a.rows_per_warp * kWarps);
    if (blocks > most) blocks = most;
    return launch_pdl(route_logits_kernel<V, T, FULL, KEYS>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, s, a);
}

template <int V, typename T>
cudaError_t launch_place(const RouteLogitsArgs& a, int num_sms, int lanes, cudaStream_t s)
{
    constexpr int size = (int)sizeof(T), bytes = V * size < 16 ? V * size : 16;
    const bool full = lanes * a.groups == 32 && a.E == 32 * V && reinterpret_cast<uintptr_t>(a.logits) % bytes == 0 &&
                      (a.T == 1 || a.stride * size % bytes == 0);
    if (a.bias) return full ? launch<V, T, true, kByBiased>(a, num_sms, s) : launch<V, T, false, kByBiased>(a, num_sms, s);
    if (a.groups > 1 && a.group_top == 2)
        return full ? launch<V, T, true, kByPairs>(a, num_sms, s) : launch<V, T, false, kByPairs>(a, num_sms, s);
    return full ? launch<V, T, true, kByLogit>(a, num_sms, s) : launch<V, T, false, kByLogit>(a, num_sms, s);
}

}  // namespace

// The launcher of one type of logits (each is compiled by a file of its own, beside the
// others).
template <typename T>
cudaError_t launch_route_logits_of(const RouteLogitsArgs& a, int num_sms, cudaStream_t s)
{
    if (a.T == 0) return cudaSuccess;
    int lanes = 32 / a.groups;
    while (lanes & (lanes - 1)) lanes &= lanes - 1;
    const int per_lane = (a.E / a.groups + lanes - 1) / lanes;
    if (per_lane <= 1) return launch_place<1, T>(a, num_sms, lanes, s);
    if (per_lane <= 2) return launch_place<2, T>(a, num_sms, lanes, s);
    if (per_lane <= 4) return launch_place<4, T>(a, num_sms, lanes, s);
    if (per_lane <= 8) return launch_place<8, T>(a, num_sms, lanes, s);
    if (per_lane <= 16) return launch_place<16, T>(a, num_sms, lanes, s);
    return cudaErrorInvalidValue;
}

}  // namespace moe
