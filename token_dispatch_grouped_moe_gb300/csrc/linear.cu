// linear.cu -- the grouped product with an epilogue on the 5th-generation tensor
// cores (bf16 or fp16 operands, fp32 sums):
//
//   out[p, n] = act(sum_k a[p, k] w[g, k, n] + bias[g, n]) + residual[p, n]
//
// for the rows p of group g (offsets[g] <= p < offsets[g + 1]), or of one group.
//
// The tile is taken the other way round, D[n, p] = sum_k w[k, n] a[p, k]: 128
// columns n of the output are the M of an MMA and the rows p its N, which may be
// any multiple of 16 up to BN. So a group's rows are not padded to a tile of 128:
// the loads, the MMAs and the epilogue take the rows that there are, and one
// form serves a token of a decode step and a prefill. The operands are read as
// they lie in memory: w with contiguous n (an M-major operand) or contiguous k.
//
// The tensor cores' running sum is cut every 512 k, whatever the output's type: the epilogue
// warps add each stretch to fp32 registers while the next one is computed into the other
// TMEM buffer. The sum in TMEM is rounded towards zero at every step, so a long one drifts:
// of the result, sums that cancel / sums of one sign, 512 k 4.8e-7 / 0.7e-6 in bf16 (K =
// 4096) and 6.5e-7 / 2.5e-6 in fp16 (K = 2048; an fp32 sum of its products one by one 6e-7); 1024 k
// 1.0e-6 / 1.7e-6 and 1.3e-6 / 5.5e-6; 2048 k 2.1e-6 / 4.3e-6 and 2.5e-6 / 11e-6. Longer
// stretches are faster where the tensor cores bound the product (16384 rows of 8 experts 4096
// -> 14336, sustained, us: 512 k 1233, 1024 1167, 2048 1152; 8192 x 4096 x 4096 with
// residual 188, 175, 177), but no sum in fp32.
//
// Kernel shape: one CTA per SM (384 threads; the form for up to 32 rows 256, two of which
// fit on an SM), persistent over (group, row tile, n tile) tiles computed from the group
// offsets:
//   warps 0..7  epilogue: warp w reads TMEM lanes 32 (w mod 4) .. + 31 (columns n,
//               one a thread) and half of the rows (up to 32 rows: warps 0..3, all);
//   the others  TMEM allocator and MMA issuer; three TMA producers, every third K
//               block each: the wait, the barrier's bytes and three to six copies take
//               one thread 650-850 cycles, more than the block's MMAs (with sums of 2048 k,
//               where it showed most: one producer 8192 x 4096 x 4096 161 us instead of 150).
// CTA pairs (PAIR): a 2-CTA cluster shares one tcgen05.mma.cta_group::2 of 256
// columns n, each CTA staging its 128 of them and half of the rows; both CTAs'
// boxes complete on rank 0's barrier, rank 0 issues, its commits arrive in both CTAs,
// and both CTAs' epilogue warps release a TMEM buffer on rank 0. A pair takes 256 rows, or
// 128: as many MMAs a block as one CTA with twice the columns, its 16 KB of weights and 8 of
// rows leave room for nine stages instead of six, and a block takes 380-460 cycles.
// When the tiles do not fill the SMs evenly (few rows), K is cut: the blocks of the
// tiles that are left over, end to end, go to the CTAs in equal runs; each CTA writes
// the sums of a tile that it has only a part of to the workspace and takes a ticket,
// and the last one adds the parts in the order of their blocks (so the result does
// not depend on which came last) and runs the epilogue. No CTA waits for another.
// Every wait is bounded (ptx.cuh).
//
// What bounds it (one GB300; us in about a second of passes, at the power cap, and in 20):
//   - many rows: the tensor cores, and the reading of their sums every 512 k. 8192 x 4096 x
//     4096 with bias and residual 188 (1460 TFLOP/s) and 165 (1660), the tensor pipe busy 74%
//     of the cycles; 16384 rows of 8 experts 4096 -> 14336 with gelu_tanh 1280 (1500) and 1110
//     (1730); a plain library product reaches 1902 TFLOP/s for a moment and 1712 at the
//     power cap. A block's 512 cycles of MMAs are also what shared memory takes to pass its
//     operands in and out (128 bytes a cycle), so one CTA per MMA, which passes twice as
//     much for the same sums, takes half as long again (8192 x 4096 x 4096 219 for 147 without
//     an epilogue): pairs, wherever there are tiles enough. 8192 x 4096 x 256 with fp32
//     outputs 20 (one CTA 22, pairs of 256 rows 25).
//   - few rows: the weights' bytes. 789 tokens' top 8 of 64 experts 3584 -> 2560 190
//     (6.6 TB/s; one CTA 196, pairs of 256 rows 198), 128 tokens' top 6 2048 -> 1408 61 (6.1).
//   - one token, 4096 -> 14336: 23.5, of which 17 stream the weights at 7 TB/s; the
//     first loads, the last tile's epilogue and the launch are the rest.
//   - in between (100 to 1000 rows of one group): the join of cut tiles, or tiles that do
//     not fill the SMs: 400 x 4096 x 4096 18.2 (21 on one CTA), 256 x 14336 x 4096 35 (41).
#include <atomic>
#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.cuh"
#include "ops.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int BM = 128;             // columns of the output that a CTA has of a tile
constexpr int BK = kLinearBK;
constexpr int W_BYTES = BM * BK * 2;
constexpr int PRODUCERS = 3;
// registers with 8 epilogue warps: 12 warps are launched with 168 each; the epilogue
// warps (up to 128 sums and 64 loads in flight) take 216 once the other warpgroup has
// gone down to 72 (8 * 216 + 4 * 72 = 12 * 168)
constexpr int EPI_REGS = 216;
constexpr int OTHER_REGS = 72;
constexpr int MAX_GROUPS = 256;
constexpr int BAND = 16;            // row tiles that are taken together
constexpr int STRETCH = 8;          // K blocks between two reads of the tensor cores' sums

// BN: rows of a tile at most. The form for few rows (32) leaves room for a second
// CTA on its SM: that of the next kernel, which gets ready meanwhile.
template <bool PAIR, int BN>
struct Cfg {
    static constexpr int EPI_WARPS = BN <= 32 ? 4 : 8;
    static constexpr int HALF = BN / (EPI_WARPS / 4);           // rows of an epilogue thread
    static constexpr int NUM_THREADS = 32 * EPI_WARPS + 128;
    static constexpr int CTAS = BN <= 32 ? 2 : 1;               // that fit on an SM
    static constexpr int A_ROWS = PAIR ? BN / 2 : BN;           // rows that a CTA stages
    static constexpr int STAGE_BYTES = W_BYTES + A_ROWS * BK * 2;
    static constexpr int STAGES = BN <= 32 ? 5 : STAGE_BYTES == 24 * 1024 ? 9 : 6;
    static constexpr int TMEM_COLS = 2 * BN;                    // two buffers
    static constexpr int TILE_N = PAIR ? 2 * BM : BM;           // columns of one work item
    static constexpr int ROW_STEP = PAIR ? 32 : 16;             // the MMA's N is a multiple of this
};

struct Tile {
    int g, row0, rows, n0;
};

// The schedule: the first `full` tiles whole, round robin over the CTAs; the K
// blocks of the rest, end to end, in `segments` equal runs, one a CTA. A run
// that begins or ends inside a tile computes a part of its sums.
struct Plan {
    int tiles, full, segments;
    int part_rows;   // rows a part has room for: those of the fullest tile, in 32s
};

template <int STAGES>
struct SmemTail {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];                 // a stretch's sums are there
    uint64_t tempty[2];                // they are read (a pair: by both CTAs, on rank 0's)
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int last;                          // cut tiles: this CTA took the tile's last ticket
    int most_rows;                     // rows of the fullest tile
    int groups;                        // that have rows
    int tile_start[MAX_GROUPS + 1];    // row tiles before each group
    int offsets[MAX_GROUPS + 1];
};

template <bool PAIR, int BN>
constexpr size_t smem_bytes()
{
    using C = Cfg<PAIR, BN>;
    return 1024 + (size_t)C::STAGES * C::STAGE_BYTES + sizeof(SmemTail<C::STAGES>);
}
static_assert(smem_bytes<false, 32>() <= 113 * 1024 && smem_bytes<false, 128>() <= 227 * 1024 &&
                  smem_bytes<true, 128>() <= 227 * 1024 && smem_bytes<true, 256>() <= 227 * 1024, "shared memory");

// A group's rows are spread evenly over its row tiles.
template <int STEP>
__device__ __forceinline__ int rows_per_tile(int rows, int tiles)
{
    return (int)(((unsigned)(rows + tiles - 1) / (unsigned)tiles + STEP - 1) / STEP * STEP);
}

// Tile w: group-major; within a group, bands of BAND row tiles, in a band n tile by
// n tile (neighbouring CTAs share a tile of w, and a band's rows stay in L2 while
// all of w passes).
template <int TILE_N, int STEP>
__device__ __forceinline__ Tile decode_tile(int w, int n_tiles, const int* ts, const int* offs, int G)
{
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ts[mid] * n_tiles <= w) lo = mid; else hi = mid;
    }
    Tile r;
    r.g = lo;
    const int mt = ts[lo + 1] - ts[lo];
    unsigned tl = (unsigned)(w - ts[lo] * n_tiles);
    const unsigned band = tl / (unsigned)(BAND * n_tiles);
    tl -= band * (unsigned)(BAND * n_tiles);
    const unsigned in_band = min((unsigned)BAND, mt - band * BAND);
    const unsigned n_tile = tl / in_band;
    const int m_tile = (int)(band * BAND + tl - n_tile * in_band);
    const int per = rows_per_tile<STEP>(offs[lo + 1] - offs[lo], mt);
    r.row0 = offs[lo] + m_tile * per;
    r.rows = min(per, offs[lo + 1] - r.row0);
    r.n0 = (int)n_tile * TILE_N;
    return r;
}

struct Piece {
    int tile, kb0, kb1;
};

struct Walk {   // make_plan keeps the products below 2^32
    uint32_t tile, step, full, k_blocks, pos, end;

    __device__ __forceinline__ Walk(const Plan& p, int unit, int n_units, int k_blocks_)
        : tile(unit), step(n_units), full(p.full), k_blocks(k_blocks_), pos(0), end(0)
    {
        if (unit < p.segments) {
            const uint32_t total = (uint32_t)(p.tiles - p.full) * k_blocks;
            pos = total * (uint32_t)unit / (uint32_t)p.segments;
            end = total * (uint32_t)(unit + 1) / (uint32_t)p.segments;
        }
    }

    __device__ __forceinline__ bool next(Piece& p)
    {
        if (tile < full) {
            p = {(int)tile, 0, (int)k_blocks};
            tile += step;
            return true;
        }
        if (pos >= end) return false;
        const uint32_t q = pos / k_blocks, kb0 = pos - q * k_blocks;
        p = {(int)(full + q), (int)kb0, (int)min(k_blocks, kb0 + (end - pos))};
        pos += (uint32_t)p.kb1 - kb0;
        return true;
    }
};

// The parts of tile q of the segments' tiles: the first segment that holds
// blocks of it, and how many do. Segment c keeps a part that begins with its
// tile in slot 2c + 1, one that begins inside it in slot 2c.
__device__ __forceinline__ int first_part(const Plan& p, int q, int k_blocks, int& parts)
{
    const uint32_t total = (uint32_t)(p.tiles - p.full) * (uint32_t)k_blocks;
    auto segment_of = [&](uint32_t block) { return linear_segment_of(block, (uint32_t)p.segments, total); };
    const int first = segment_of((uint32_t)q * (uint32_t)k_blocks);
    parts = segment_of((uint32_t)(q + 1) * (uint32_t)k_blocks - 1) - first + 1;
    return first;
}

// The plan with the least estimated time (linear_candidate), one candidate a lane; the
// warp calls it together.
template <bool PAIR, int BN>
__device__ __forceinline__ Plan make_plan(int tiles, int w_tiles, int rows, int k_blocks, int n_units, int lane)
{
    const LinearCandidate c = linear_candidate(linear_form_of(PAIR, BN), lane, tiles, w_tiles, rows, k_blocks, n_units);
    const int best = (int)(__reduce_min_sync(0xffffffffu, linear_candidate_key(c, lane)) & 31u);
    return Plan{tiles, __shfl_sync(0xffffffffu, c.full, best), __shfl_sync(0xffffffffu, c.segments, best),
                linear_part_rows(rows)};
}

template <int WARPS>
__device__ __forceinline__ void epilogue_barrier()   // the epilogue warps only
{
    asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory");
}

// Adds this thread's rows c < rows of the parts s0 .. s1 - 1 of a tile to acc, in
// order: a row of a part is BM floats, one a column (src: this thread's column of the
// row 0 of slot 2 first). ROWS rows of PARTS parts are in flight together (each a
// trip to L2): all that the registers hold.
template <int HALF, int ROWS, int PARTS>
__device__ __forceinline__ void add_parts(float (&acc)[HALF], const float* src, int rows, int begin, int end,
                                          int64_t stride)
{
    // the first part begins with the tile, the others inside it (first_part)
    auto slot = [&](int s) { return (int64_t)(s == 0 ? 1 : 2 * s) * stride; };
#pragma unroll
    for (int c = 0; c < (ROWS < 32 ? ROWS : HALF); c += ROWS) {
        if (c >= rows) break;
        for (int s0 = begin; s0 < end; s0 += PARTS) {
            // (no branch between the loads, which would make them wait for one another: rows
            // past the last are read as they are, of this part or the next; parts past the
            // last are the last again)
            float v[PARTS][ROWS];
#pragma unroll
            for (int s = 0; s < PARTS; ++s) {
                const float* part = src + slot(min(s0 + s, end - 1));
#pragma unroll
                for (int i = 0; i < ROWS; ++i) v[s][i] = __ldcg(part + (c + i) * BM);
            }
#pragma unroll
            for (int s = 0; s < PARTS; ++s)
                if (s0 + s < end) {
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) acc[c + i] += v[s][i];
                }
        }
    }
}

// 2^x, within 2^-22 of itself; 0 below 2^-126
__device__ __forceinline__ float exp2_near(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max_or_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// x (1 + erf(x / sqrt 2)) / 2 = max(x, 0) - |x| q, q = erfc(|x| / sqrt 2) / 2 = p(t) t
// e^(-x^2 / 2), t = 1 / (1 + c |x|). p has the least largest relative error of the
// polynomials of its degree over |x| <= 14 (Remez's exchange, in 40 digits): so the result is
// near relative to itself also where it is small, at x = -12 as well as at -1, and not
// relative to erfc's 1 only. For fp32 outputs (FINE) degree 7, 1.05e-7, and the
// exponent's rounding made good by what it left out: within 16 * 2^-23. For 16 bits, whose
// half steps are 2^-11 and more, degree 5, 4.0e-6, and 2^-15 at most: a prefill of 16384 rows,
// 8 experts 4096 -> 14336, takes 1244 us, with the finer one 1410, with erfcf 2180.
template <bool FINE>
__device__ __forceinline__ float gelu(float x)
{
    constexpr float kScale = -0.72134752044448170368f;   // -log2(e) / 2
    float q;
    if constexpr (FINE) {
        constexpr float kScaleLow = (float)(-0.72134752044448170368 - (double)kScale);
        const float a = fminf(fabsf(x), 20.0f);          // (from there on q is 0)
        const float t = __fdividef(1.0f, fmaf(0.305f, a, 1.0f));
        q = fmaf(0.036699183f, t, -0.15298827f);
        q = fmaf(q, t, 0.18571681f);
        q = fmaf(q, t, -0.03797674f);
        q = fmaf(q, t, 0.121021636f);
        q = fmaf(q, t, 0.10342088f);
        q = fmaf(q, t, 0.12246682f);
        q = fmaf(q, t, 0.121639736f);
        const float square = a * a, n = square * kScale;
        const float left = fmaf(square, kScale, -n) + fmaf(fmaf(a, a, -square), kScale, square * kScaleLow);
        q = q * t * (exp2_near(n) * fmaf(left, 0.69314718f, 1.0f));
    } else {
        const float t = __fdividef(1.0f, fmaf(0.308f, fabsf(x), 1.0f));
        q = fmaf(-0.0754302f, t, 0.18961859f);
        q = fmaf(q, t, 0.007272298f);
        q = fmaf(q, t, 0.13653392f);
        q = fmaf(q, t, 0.118881136f);
        q = fmaf(q, t, 0.12312271f);
        q = q * t * exp2_near(x * x * kScale);
    }
    return fmaf(-fminf(fabsf(x), 1e30f), q, max_or_nan(x, 0.0f));   // (an infinity times q = 0 is no number)
}

// 0.5 x (1 + tanh(u)) = x / (1 + e^(-2u)), u = sqrt(2/pi) (x + 0.044715 x^3)
__device__ __forceinline__ float gelu_tanh(float x)
{
    const float u2 = x * fmaf(0.071354816272600125f, x * x, 1.5957691216057308f);
    return __fdividef(x, 1.0f + __expf(-u2));
}

__device__ __forceinline__ float silu_of(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

template <bool FINE, int N>
__device__ __forceinline__ void activate(float (&v)[N], int act)
{
    switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];   // keeps a NaN
        break;
    case MOE_ACT_SILU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = silu_of(v[i]);
        break;
    case MOE_ACT_GELU:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = gelu<FINE>(v[i]);
        break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = gelu_tanh(v[i]);
        break;
    default: break;
    }
}

template <bool PAIR>
__device__ __forceinline__ void load_2d(uint32_t dst, const void* map, int c0, int c1, uint32_t bar)
{
    if (PAIR) tma_load_2d_pair(dst, map, c0, c1, bar); else tma_load_2d(dst, map, c0, c1, bar);
}

template <bool PAIR>
__device__ __forceinline__ void load_3d(uint32_t dst, const void* map, int c0, int c1, int c2, uint32_t bar)
{
    if (PAIR) tma_load_3d_pair(dst, map, c0, c1, c2, bar); else tma_load_3d(dst, map, c0, c1, c2, bar);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A value's bits in a register, and what they are.
__device__ __forceinline__ uint32_t load_raw(const float* p)
{
    uint32_t r;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(r) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t load_raw(const void* p)
{
    uint32_t r;
    asm volatile("ld.global.u16 %0, [%1];" : "=r"(r) : "l"(p) : "memory");
    return r;
}
template <typename T>
__device__ __forceinline__ float of_raw(uint32_t r)
{
    if constexpr (sizeof(T) == 4) return __uint_as_float(r);
    else if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)r));
    else return __uint_as_float(r << 16);
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// The rows of this CTA's part of a tile of the residual to L2, a thread a row.
template <typename OUT, int EPI_THREADS>
__device__ __forceinline__ void prefetch_residual(const LinearArgs& args, const Tile& it, uint32_t rank)
{
    const int n0 = it.n0 + (int)rank * BM, cols = min(BM, args.N - n0);
    if (cols <= 0) return;
    for (int r = threadIdx.x; r < it.rows; r += EPI_THREADS) {
        const OUT* res = static_cast<const OUT*>(args.residual) + (int64_t)(it.row0 + r) * args.residual_stride + n0;
        for (int c = 0; c < cols; c += 128 / (int)sizeof(OUT)) prefetch_l2(res + c);
        prefetch_l2(res + cols - 1);
    }
}

template <typename OUT, bool PAIR, int BN>
__global__ void __launch_bounds__(Cfg<PAIR, BN>::NUM_THREADS, Cfg<PAIR, BN>::CTAS)
linear_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_a_small,
              const __grid_constant__ CUtensorMap tm_w, const LinearArgs args)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t tiles_addr = (raw_addr + 1023u) & ~1023u;
    using C = Cfg<PAIR, BN>;
    constexpr int EPI_WARPS = C::EPI_WARPS;
    constexpr int HALF = C::HALF;
    constexpr int STAGES = C::STAGES;
    constexpr int CG = PAIR ? 2 : 1;   // tcgen05 CTA group
    SmemTail<STAGES>* st =
        reinterpret_cast<SmemTail<STAGES>*>(smem_raw + (tiles_addr - raw_addr) + (size_t)STAGES * C::STAGE_BYTES);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = args.G;
    // a pair walks the schedule together, each CTA with its half of every tile's columns
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const int unit = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int n_units = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&st->full[s]), 1);
            mbar_init(smem_u32(&st->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&st->tfull[a]), 1);
            mbar_init(smem_u32(&st->tempty[a]), CG * EPI_WARPS);
        }
        mbar_init(smem_u32(&st->drain), 1);
        st->abort = 0;
        fence_barrier_init();
    }
    if (warp == EPI_WARPS && lane == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_a_small);
        tma_prefetch_desc(&tm_w);
    }
    if (warp == EPI_WARPS + 1) {
        tmem_alloc<CG>(smem_u32(&st->tmem_base), C::TMEM_COLS);
        tmem_relinquish<CG>();
    }
    // a dense product's schedule does not wait for the kernel before it
    if (args.offsets) pdl_wait();
    if (warp == 0) {
        // the row tiles before each group, a lane a run of up to PER groups; offsets that
        // decrease or leave [0, R] are reported and give no tiles at all, so no row
        // outside the operands is touched
        constexpr int PER = MAX_GROUPS / 32;
        const int per = (G + 31) / 32, g0 = lane * per;
        int off[PER + 1];
#pragma unroll
        for (int i = 0; i <= PER; ++i) {
            off[i] = g0 + i ? args.R : 0;
            if (args.offsets && i <= per && g0 + i <= G) off[i] = args.offsets[g0 + i];
        }
        bool good = true;
        int tiles[PER], sum = 0;
        int most = 0, groups = 0;   // rows of the fullest tile; groups that have rows
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            tiles[i] = 0;
            if (i < per && g0 + i < G) {
                good = good && off[i] >= 0 && off[i] <= off[i + 1] && off[i + 1] <= args.R;
                const int rows = good ? off[i + 1] - off[i] : 0;
                if (rows) {
                    tiles[i] = (int)((unsigned)(rows + args.tile_rows - 1) / (unsigned)args.tile_rows);
                    most = max(most, rows_per_tile<C::ROW_STEP>(rows, tiles[i]));
                    sum += tiles[i];
                    ++groups;
                }
            }
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        int before = incl - sum;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i < per && g0 + i < G) {
                st->offsets[g0 + i] = off[i];
                st->tile_start[g0 + i] = before;
                before += tiles[i];
                if (g0 + i == G - 1) st->offsets[G] = off[i + 1];
            }
        good = __all_sync(0xffffffffu, good);
        most = __reduce_max_sync(0xffffffffu, most);
        groups = __reduce_add_sync(0xffffffffu, groups);
        const int all = __shfl_sync(0xffffffffu, incl, 31);
        if (lane == 0) {
            st->tile_start[G] = good ? all : 0;
            st->most_rows = most;
            st->groups = groups;
            if (!good) report_error(args.err, MOE_DEV_ERR_BOUNDS);
        }
    }
    tc_fence_before();
    // a pair: both CTAs' barriers are initialised before either signals the other's
    if (PAIR) cluster_sync(); else __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = st->tmem_base;
    const int n_tiles = (args.N + C::TILE_N - 1) / C::TILE_N;
    const int k_blocks = (args.K + BK - 1) / BK;
    const Plan plan = make_plan<PAIR, BN>(st->tile_start[G] * n_tiles, st->groups * n_tiles, st->most_rows, k_blocks, n_units, lane);
    volatile int* abort = &st->abort;
    auto decode = [&](int tile) {
        return decode_tile<C::TILE_N, C::ROW_STEP>(tile, n_tiles, st->tile_start, st->offsets, G);
    };

    if (warp >= EPI_WARPS) {
        if constexpr (EPI_WARPS == 8) setmaxnreg_dec<OTHER_REGS>();
        if (warp != EPI_WARPS + 1) {
            // ============================ TMA producers ============================
            if (lane == 0) {
                const int turn = max(0, warp - EPI_WARPS - 1);   // of the K blocks, counted over all pieces
                int stage = turn;
                uint32_t phase = 0;
                int issued = 0;
                int skip = turn;                                 // blocks before this producer's next one
                bool ok = true;
                Walk walk(plan, unit, n_units, k_blocks);
                Piece pc;
                bool more = walk.next(pc);
                Tile it = more ? decode(pc.tile) : Tile{0, 0, 0, 0};
                if (!args.offsets) pdl_wait();
                for (bool first = true; ok && more; more = walk.next(pc), first = false) {
                    if (!first) it = decode(pc.tile);
                    // this CTA's rows: boxes of 128, then of 32 up to the last one that the MMA
                    // reads (a pair: each CTA its half of them)
                    const int rows = PAIR ? (it.rows + 31) / 32 * 16 : it.rows;
                    const int row0 = it.row0 + (int)rank * rows;
                    const int n0 = it.n0 + (int)rank * BM;
                    const int large = rows / kLinearRowBox;
                    const int small = (rows - large * kLinearRowBox + kLinearRowBoxSmall - 1) / kLinearRowBoxSmall;
                    const uint32_t bytes = W_BYTES + (uint32_t)(large * kLinearRowBox + small * kLinearRowBoxSmall) * BK * 2;
                    int kb = pc.kb0 + skip;
                    for (; kb < pc.kb1; kb += PRODUCERS) {
                        if (!mbar_wait(smem_u32(&st->empty[stage]), phase ^ 1u, abort, args.err)) {
                            ok = false;
                            break;
                        }
                        uint32_t full = smem_u32(&st->full[stage]);
                        const uint32_t w_dst = tiles_addr + stage * C::STAGE_BYTES;
                        uint32_t a_dst = w_dst + W_BYTES;
                        if (rank == 0) mbar_arrive_expect_tx(full, CG * bytes);
                        if (PAIR) full = mapa_shared(full, 0);
                        if (args.w_nk) {
                            load_3d<PAIR>(w_dst, &tm_w, kb * BK, n0, it.g, full);
                        } else {
                            load_3d<PAIR>(w_dst, &tm_w, n0, kb * BK, it.g, full);
                            load_3d<PAIR>(w_dst + W_BYTES / 2, &tm_w, n0 + 64, kb * BK, it.g, full);
                        }
                        int row = row0;
                        for (int i = 0; i < large; ++i, row += kLinearRowBox, a_dst += kLinearRowBox * BK * 2)
                            load_2d<PAIR>(a_dst, &tm_a, kb * BK, row, full);
                        for (int i = 0; i < small; ++i, row += kLinearRowBoxSmall, a_dst += kLinearRowBoxSmall * BK * 2)
                            load_2d<PAIR>(a_dst, &tm_a_small, kb * BK, row, full);
                        ++issued;
                        if ((stage += PRODUCERS) >= STAGES) { stage -= STAGES; phase ^= 1u; }
                    }
                    skip = kb - pc.kb1;
                }
                if (!PAIR && !ok) {
                    // drain: wait (bounded) for the loads still in flight
                    for (int i = 0; i < min(issued, (STAGES + PRODUCERS - 1) / PRODUCERS); ++i) {
                        if ((stage -= PRODUCERS) < 0) { stage += STAGES; phase ^= 1u; }
                        mbar_wait_drain(smem_u32(&st->full[stage]), phase);
                    }
                }
            }
            __syncwarp();
        } else {
            // ============================ MMA issuer ==============================
            // the whole warp walks the pieces and waits (uniform control flow, so the
            // descriptors stay in uniform registers); one elected lane issues (a
            // pair: of the rank-0 CTA, for both)
            const uint32_t leader = elect_one_sync();
            // w with contiguous n: 64 n x 8 k atoms, the second 64 n 8 KB on, a K step of
            // 16 rows of 128 bytes; with contiguous k (as a): 32 bytes along the row
            const uint64_t w_desc = args.w_nk ? smem_desc_sw128(tiles_addr, 16, 1024)
                                              : smem_desc_sw128(tiles_addr, W_BYTES / 2, 1024);
            const uint64_t w_step = args.w_nk ? 2 : 16 * 128 / 16;
            const uint64_t a_desc = smem_desc_sw128(tiles_addr + W_BYTES, 16, 1024);
            const uint32_t fmt = args.fp16 ? 0u : 1u;
            const uint32_t idesc0 =
                (1u << 4) | (fmt << 7) | (fmt << 10) | ((args.w_nk ? 0u : 1u) << 15) | ((C::TILE_N >> 4) << 24);
            int stage = 0;
            uint32_t phase = 0;
            int buf = 0;
            uint32_t buf_phase = 0;
            bool ok = true;
            bool any = false;
            bool ready = false;    // the next block is known to be there
            Walk walk(plan, unit, n_units, k_blocks);
            // (the limit of the waits below is not to count the kernel before this one, for which
            // the producers wait)
            if (!args.offsets) pdl_wait();
            for (Piece pc; ok && rank == 0 && walk.next(pc);) {
                const Tile it = decode(pc.tile);
                const uint32_t idesc =
                    idesc0 | ((uint32_t)((it.rows + C::ROW_STEP - 1) / C::ROW_STEP * C::ROW_STEP >> 3) << 17);
                int in = 0;   // of the stretch
                for (int kb = pc.kb0; kb < pc.kb1; ++kb) {
                    const bool opens = in == 0;
                    ok = __all_sync(0xffffffffu,
                                    (ready || mbar_wait(smem_u32(&st->full[stage]), phase, abort, args.err)) &&
                                        (!opens || mbar_wait<PAIR, PAIR>(smem_u32(&st->tempty[buf]), buf_phase ^ 1u,
                                                                         abort, args.err)));
                    if (!ok) break;
                    tc_fence_after();
                    const bool closes = ++in == STRETCH || kb == pc.kb1 - 1;
                    const int at_stage = stage;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    // whether the next block is there, asked before this one's MMAs
                    ready = mbar_test(smem_u32(&st->full[stage]), phase);
                    if (leader) {
                        const uint32_t d = tmem_base + buf * BN;
                        const uint64_t at = (uint64_t)(at_stage * (C::STAGE_BYTES >> 4));
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            tc_mma_f16<CG>(d, w_desc + at + w_step * kk, a_desc + at + 2 * kk, idesc,
                                           !opens || kk != 0 ? 1u : 0u);
                        tc_commit<CG>(smem_u32(&st->empty[at_stage]));
                        if (closes) tc_commit<CG>(smem_u32(&st->tfull[buf]));
                    }
                    __syncwarp();
                    any = true;
                    if (closes) {
                        in = 0;
                        if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
                    }
                }
            }
            if (!ok && any && leader) {
                // drain: every MMA issued so far must finish before TMEM is freed
                if (PAIR) tc_commit_pair_local(smem_u32(&st->drain));
                else tc_commit(smem_u32(&st->drain));
                mbar_wait_drain(smem_u32(&st->drain), 0);
            }
            __syncwarp();
        }
        if (!args.offsets) pdl_wait();
        pdl_launch_dependents();
    } else {
        if constexpr (EPI_WARPS == 8) setmaxnreg_inc<EPI_REGS>();
        if (!args.offsets) pdl_wait();
        pdl_launch_dependents();
        // ============================== epilogue ==============================
        const int c0 = (warp >> 2) * HALF;             // this thread's rows of the tile (from)
        const uint32_t t_row = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + c0;
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        // after an abort every epilogue warp still walks all pieces, without waiting
        // for the tensor cores, so that the barriers below stay matched
        Walk walk(plan, unit, n_units, k_blocks);
        for (Piece pc; walk.next(pc);) {
            const Tile it = decode(pc.tile);
            const int rows = it.rows - c0;             // of them there are so many
            const int n = it.n0 + (int)rank * BM + (warp & 3) * 32 + lane;
            float bias = 0.0f;
            if (args.bias && n < args.N) {
                const int64_t at = (int64_t)it.g * args.N + n;
                bias = args.bias_f32 ? __ldg(static_cast<const float*>(args.bias) + at)
                       : args.fp16   ? __half2float(static_cast<const __half*>(args.bias)[at])
                                     : __bfloat162float(static_cast<const __nv_bfloat16*>(args.bias)[at]);
            }
            const bool whole = pc.kb1 - pc.kb0 == k_blocks;
            // without an activation the sums begin with the residual, whose loads pass while
            // the tensor cores work; else it is added at the end, from L2, where it is asked
            // for now (8192 x 4096 x 4096, sums of 2048 k, us: 149 without a residual, 168 with;
            // silu 158 and 184)
            const bool early = args.residual && whole && args.act == MOE_ACT_NONE;
            if (args.residual && !early && pc.kb1 == k_blocks) prefetch_residual<OUT, 32 * EPI_WARPS>(args, it, rank);
            const int q = pc.tile - plan.full;         // of a cut tile: its number and parts
            int parts = 0;
            const int first = whole ? 0 : first_part(plan, q, k_blocks, parts);
            float acc[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) acc[i] = 0.0f;
            if (early && n < args.N && rows > 0) {
                const OUT* res = static_cast<const OUT*>(args.residual) + (int64_t)(it.row0 + c0) * args.residual_stride + n;
                uint32_t raw[HALF];   // all loads before the first use, without a branch between them
#pragma unroll
                for (int c = 0; c < HALF; ++c) raw[c] = load_raw(res + min(c, rows - 1) * args.residual_stride);
#pragma unroll
                for (int c = 0; c < HALF; ++c) acc[c] = of_raw<OUT>(raw[c]);
            }
            for (int kb = pc.kb0; kb < pc.kb1 && ok; kb += STRETCH) {
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&st->tfull[buf]), buf_phase, abort, args.err));
                if (!ok) break;
                tc_fence_after();
                const uint32_t t = t_row + buf * BN;
#pragma unroll
                for (int c = 0; c < HALF; c += 32) {
                    if (c < rows) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(t + c, v);
                        tc_wait_ld_for(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[c + i] += __uint_as_float(v[i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && rank != 0) mbar_arrive_remote_tmem(mapa_shared(smem_u32(&st->tempty[buf]), 0));
                    else mbar_arrive(smem_u32(&st->tempty[buf]));
                }
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            }
            if (!whole) {
                // publish this piece's part and take a ticket; the last piece of the tile
                // adds the parts up
                const int64_t stride = (int64_t)plan.part_rows * CG * BM;
                float* base = args.part + ((int64_t)rank * plan.part_rows + c0) * BM + (warp & 3) * 32 + lane;
                float* part = base + (2 * unit + (pc.kb0 == 0)) * stride;
                if (ok) {
#pragma unroll
                    for (int c = 0; c < HALF; ++c)
                        if (c < rows) __stcg(part + c * BM, acc[c]);
                }
                epilogue_barrier<EPI_WARPS>();
                if (threadIdx.x == 0) {
                    // the barrier orders the warps' parts before this thread's fence, and the
                    // fence behind the ticket orders it before the other CTAs' parts are read
                    int last = 0;
                    __threadfence();
                    if (!*abort) {
                        int32_t* ticket = args.ticket + q * CG + rank;
                        last = atomicAdd(ticket, 1) == parts - 1;
                        if (last) *ticket = 0;   // as found, for the next call
                    }
                    __threadfence();
                    st->last = last;
                }
                epilogue_barrier<EPI_WARPS>();
                if (!st->last) continue;
                const float* src = base + 2 * first * stride;
                // the sum of two parts does not depend on their order: the other one is added
                // to this CTA's
                const int mine = unit - first;
                const int begin = parts == 2 ? 1 - mine : 0, end = parts == 2 ? 2 - mine : parts;
                if (parts != 2) {
#pragma unroll
                    for (int i = 0; i < HALF; ++i) acc[i] = 0.0f;
                }
                if (rows <= 2) add_parts<HALF, 2, 8>(acc, src, rows, begin, end, stride);
                else if (rows <= 8) add_parts<HALF, 8, 4>(acc, src, rows, begin, end, stride);
                else if (HALF == 64 && parts == 2) add_parts<HALF, HALF, 1>(acc, src, rows, begin, end, stride);
                else if (HALF == 128) add_parts<HALF, 32, 1>(acc, src, rows, begin, end, stride);
                else add_parts<HALF, 32, 2>(acc, src, rows, begin, end, stride);
            }
            if (!ok) continue;
            if (n < args.N) {
                OUT* out = static_cast<OUT*>(args.out) + (int64_t)(it.row0 + c0) * args.out_stride + n;
                const OUT* res = early ? nullptr : static_cast<const OUT*>(args.residual);
                if (res) res += (int64_t)(it.row0 + c0) * args.residual_stride + n;
                // CHUNK rows at a time (few rows: no more code is fetched than they need)
                constexpr int CHUNK = HALF <= 32 ? 4 : 32;
#pragma unroll
                for (int c = 0; c < HALF; c += CHUNK) {
                    if (c >= rows) break;
                    float v[CHUNK];
#pragma unroll
                    for (int i = 0; i < CHUNK; ++i) v[i] = acc[c + i] + bias;
                    activate<sizeof(OUT) == 4>(v, args.act);
                    if (res) {
                        uint32_t r[CHUNK];
#pragma unroll
                        for (int i = 0; i < CHUNK; ++i) r[i] = load_raw(res + min(c + i, rows - 1) * args.residual_stride);
#pragma unroll
                        for (int i = 0; i < CHUNK; ++i) v[i] += of_raw<OUT>(r[i]);
                    }
#pragma unroll
                    for (int i = 0; i < CHUNK; ++i)
                        if (c + i < rows) put(out + (c + i) * args.out_stride, v[i]);
                }
            }
        }
    }

    // ---- teardown: every role is done (or has drained after an abort)
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) {
        // after an abort, give the copies and commits already issued for this
        // CTA (some by the other CTA) time to land; then neither CTA leaves
        // while the other may still use its shared memory or TMEM
        if (threadIdx.x == 0 && *abort) sleep_ns(1000000);
        cluster_sync();
    }
    if (warp == EPI_WARPS + 1) {
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, C::TMEM_COLS);
    }
}

constexpr int kMaxDevices = 64;

template <typename OUT, bool PAIR, int BN>
cudaError_t launch(const CUtensorMap& tm_a, const CUtensorMap& tm_a_small, const CUtensorMap& tm_w, const LinearArgs& a,
                   int num_sms, cudaStream_t s)
{
    auto kern = linear_kernel<OUT, PAIR, BN>;
    constexpr size_t smem = smem_bytes<PAIR, BN>();
    if (a.tile_rows <= 0 || a.tile_rows > BN || a.tile_rows % Cfg<PAIR, BN>::ROW_STEP) return cudaErrorInvalidValue;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(PAIR ? num_sms & ~1 : num_sms));
    cfg.blockDim = dim3(Cfg<PAIR, BN>::NUM_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // asked of the runtime once per kernel and device: its shared memory, and how many
    // pairs can be resident at once (shared memory and the GPCs' SM pairs decide)
    static std::atomic<int> units[kMaxDevices];
    int n = units[dev].load(std::memory_order_acquire);
    if (n <= 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        n = num_sms;
        if (PAIR) {
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess) return e;
        }
        if (n <= 0) return cudaErrorInvalidConfiguration;
        units[dev].store(n, std::memory_order_release);
    }
    if (PAIR) cfg.gridDim = dim3((unsigned)(2 * (n < num_sms / 2 ? n : num_sms / 2)));
    cfg.numAttrs = 2;   // the occupancy query above saw the cluster shape only
    if (!PAIR) {
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
    }
    e = cudaLaunchKernelEx(&cfg, kern, tm_a, tm_a_small, tm_w, a);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename OUT>
cudaError_t launch_out(LinearForm form, const CUtensorMap& tm_a, const CUtensorMap& tm_a_small, const CUtensorMap& tm_w,
                       const LinearArgs& a, int num_sms, cudaStream_t s)
{
    switch (form) {
    case kLinearFew: return launch<OUT, false, 32>(tm_a, tm_a_small, tm_w, a, num_sms, s);
    case kLinearOne: return launch<OUT, false, 128>(tm_a, tm_a_small, tm_w, a, num_sms, s);
    case kLinearPairHalf: return launch<OUT, true, 128>(tm_a, tm_a_small, tm_w, a, num_sms, s);
    case kLinearPair: return launch<OUT, true, 256>(tm_a, tm_a_small, tm_w, a, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_linear(LinearForm form, moe_dtype out_dtype, const CUtensorMap& tm_a, const CUtensorMap& tm_a_small,
                          const CUtensorMap& tm_w, const LinearArgs& a, int num_sms, cudaStream_t s)
{
    if (a.R == 0) return cudaSuccess;
    if (a.R < 0 || a.G < 1 || a.G > MAX_GROUPS || (!a.offsets && a.G != 1)) return cudaErrorInvalidValue;
    switch (out_dtype) {
    case MOE_BF16: return launch_out<__nv_bfloat16>(form, tm_a, tm_a_small, tm_w, a, num_sms, s);
    case MOE_FP16: return launch_out<__half>(form, tm_a, tm_a_small, tm_w, a, num_sms, s);
    case MOE_FP32: return launch_out<float>(form, tm_a, tm_a_small, tm_w, a, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
