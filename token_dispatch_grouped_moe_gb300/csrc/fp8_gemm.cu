// fp8_gemm.cu -- the expert products in 8-bit floating point (e4m3) on the
// 5th-generation tensor cores, with one fp32 scale for each row's block of 128
// activations and for each 128 x 128 block of a weight:
//
//   out[p, n] = sum_b sa[p, b] sw[e, n / 128, b] sum_{k in block b} a[p, k] w[e, n, k]
//
// for the rows p of expert e (offsets[e] <= p < offsets[e + 1]). Two forms:
//   product (GATED false): out in bf16 or fp32, in dispatch order, or scaled by
//     the row's gate weight and scattered to slot[rank][token] (fp32);
//   gated (GATED true): h = silu(a W1^T) * (a W3^T) for one 128-wide slice of
//     F, requantized in the epilogue: e4m3 with a scale per row and slice.
//
// The products of one block are exact in the tensor core's fp32 accumulator up
// to its own rounding; the scales differ from block to block, so the block sums
// are multiplied by sa * sw and added in registers (fp32): every 128-wide K
// block is one MMA group (M = 128, N = 256, K = 4 x 32) into one of two TMEM
// buffers, and while the tensor cores fill one the epilogue warps fold the
// other into their accumulators.
//
// Kernel shape: one CTA per SM (384 threads), persistent over a static schedule
// of (expert, N tile, M tile) tiles computed from the group offsets:
//   warps 0..7  fold and epilogue: warp w reads TMEM lanes 32 (w mod 4) .. + 31
//               (rows) and columns 128 (w / 4) .. + 127: 128 fp32 accumulators a
//               thread;
//   warp 8      TMA producer: 4-stage ring of {A 128 x 128, B 256 x 128} bytes;
//   warp 9      TMEM allocator and MMA issuer;
//   warps 10,11 the rows' factors sa * sw of each block, into shared memory.
// CTA pairs (PAIR): a 2-CTA cluster shares one tcgen05.mma.cta_group::2 of M =
// 256; both CTAs' boxes complete on rank 0's barrier, rank 0 issues, its commit
// arrives in both CTAs, and both CTAs' fold warps release a buffer on rank 0.
// A product of few tiles takes tiles of 128 columns (BN; 64 accumulators a thread,
// a buffer given back after one trip to TMEM: 0.31-0.33 us a block, of 256 columns
// 0.39-0.43).
// When the tiles do not fill the SMs evenly (few rows), K is cut: the blocks of
// the tiles that are left over, end to end, go to the CTAs in equal runs; each
// CTA writes the fp32 sums of a tile that it has only a part of to the
// workspace and takes a ticket, and the last one adds the parts in the order of
// their blocks (so the result does not depend on which came last) and runs the
// epilogue. No CTA waits for another. Every wait is bounded (ptx.cuh).
//
// What bounds it (one GB300):
//   - many rows: the fold. A block's MMAs take 512 cycles; folding its 128 x 256
//     sums takes 256 cycles of the FMA pipe in each SM quarter and, with the trips
//     to TMEM and the barriers, 800-900 in all, of which the MMAs of the next block
//     cover theirs. 8192 x 8192 x 8192: 400-420 us, 2.6-2.75 PFLOP/s (a library
//     product without block scales: 3.6-3.8). A buffer's round trip is about 950
//     cycles from its release to the next sums (the release seen, MMAs issued, 512
//     of MMAs, the commit seen) and 700 to the next release, for two buffers. Back
//     to back the product is at the GPU's power cap as well (1350 W, 1.6 GHz); the
//     gated form, with about 4000 cycles of epilogue a tile (silu 1750, conversion
//     and stores 1200), runs at 1.97 GHz. 32768 tokens, 64 experts 2048 -> 1408, top
//     6, pass after pass: gated 1050 us; 8192 tokens, 8 experts 14336 -> 4096, top 2,
//     Zipf: product 840-850 us. Measured and not kept: pairs of sums in
//     fma.rn.f32x2 (register moves: 2.0 PFLOP/s), factors four blocks at a time, N =
//     128 MMAs with four buffers, loads of the next block asked for before the last
//     sums (spills), releases without memory order, one reciprocal for two silus,
//     and warps without rows of a tile passing its blocks on unread.
//   - few rows: the weights' bytes: 1024 tokens, 64 experts 2048 -> 1408, top 6
//     5.6 TB/s, 789 tokens 2560 -> 3584, top 8 6.2 TB/s (0.83, 0.92 of a copy).
//   - one token: latency (11 us for 6 experts 1408 -> 2048: the first loads land
//     5 us after the previous kernel's end) and, on wide experts, the last run's
//     tail (8 experts 4096 -> 14336, top 2: 54 us for 235 MB).
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int BM = 128;
constexpr int BK = kFp8Block;      // one scale block of K = one 128-byte swizzle span
constexpr int A_BYTES = BM * BK;   // 16 KB
constexpr int FOLD_WARPS = 8;
constexpr int FOLD_THREADS = 32 * FOLD_WARPS;
constexpr int FACTOR_WARPS = 2;
constexpr int TILE_SLOTS = 4;      // the factor warps are at most two blocks, so two pieces, ahead
constexpr int NUM_THREADS = FOLD_THREADS + 128;
// registers: 12 warps are launched with 168 each; the fold warps (128
// accumulators, two 32-column loads in flight) take 216 once the other
// warpgroup has gone down to 72 (8 * 216 + 4 * 72 = 12 * 168)
constexpr int FOLD_REGS = 216;
constexpr int OTHER_REGS = 72;
constexpr int MAX_GROUPS = 256;

// One CTA per MMA (PAIR false): a stage holds 128 rows of A and 256 of B. A CTA
// pair (tcgen05 cta_group::2): one MMA of 256 x 256 over both CTAs, each staging
// its 128 rows of A and half of B's, so a third less comes from L2 per block.
// BN is the MMA's N (gated: 128 columns of W1 and 128 of W3, interleaved by 64):
// 256, or 128 for a product whose tiles of 128 all find an SM (product_form in
// api_fp8.cu).
template <bool PAIR, int BN>
struct Cfg {
    static constexpr int B_ROWS = PAIR ? BN / 2 : BN;
    static constexpr int STAGE_BYTES = A_BYTES + B_ROWS * BK;   // 48 KB or 32 KB
    static constexpr int STAGES = STAGE_BYTES == 48 * 1024 ? 4 : 6;
    static constexpr int TMEM_COLS = 2 * BN;                    // two buffers
    static constexpr int TILE_ROWS = PAIR ? 2 * BM : BM;        // rows of one work item
    static constexpr uint32_t IDESC = idesc_e4m3_f32(TILE_ROWS, BN);
};

struct Tile {
    int g, row0, rows, n_tile;
};

// The schedule: the first `full` tiles whole, round robin over the CTAs; the K
// blocks of the rest, end to end, in `segments` equal runs, one a CTA. A run
// that begins or ends inside a tile computes a part of its sums.
struct Plan {
    int tiles, full, segments;
    int part_rows;   // rows a part has room for: those of the fullest tile
};

template <int STAGES>
struct SmemTail {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];                 // a block's sums and its factors are there
    uint64_t tempty[2];                // the sums are read (a pair: by both CTAs, on rank 0's)
    uint64_t ffree[2];                 // the factors are read
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int last;                          // cut tiles: this CTA took the tile's last ticket
    int most_rows;                     // rows of the fullest tile
    int tile_start[MAX_GROUPS + 1];    // tiles before each group
    int offsets[MAX_GROUPS + 1];
    Tile tile[TILE_SLOTS];             // the pieces' tiles, decoded by a factor warp
    float2 factor[2][BM];              // sa * sw of each row: column halves (gated: W1 and W3)
    float amax[2][2][BM];              // gated: [piece parity][column half][row]
    uint4 stage_out[FOLD_WARPS][32 * 4];   // 64 bytes of a fold warp's 32 rows, on their way out
};
template <bool PAIR, int BN>
constexpr size_t smem_bytes()
{
    using C = Cfg<PAIR, BN>;
    return 1024 + (size_t)C::STAGES * C::STAGE_BYTES + sizeof(SmemTail<C::STAGES>);
}
static_assert(smem_bytes<false, 256>() <= 227 * 1024 && smem_bytes<true, 256>() <= 227 * 1024 &&
                  smem_bytes<false, 128>() <= 227 * 1024, "shared memory");

// Tile w: tiles go expert-major, then N tile, then M tile (neighbouring CTAs
// share the weights of an N tile in L2). This CTA's rows start `sub` rows into
// the tile (a pair's rank 1: 128) and may be none (rows <= 0).
template <int TILE_ROWS>
__device__ __forceinline__ Tile decode_tile(int w, int n_tiles, const int* ts, const int* offs, int G, int sub)
{
    Tile r;
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ts[mid] * n_tiles <= w) lo = mid; else hi = mid;
    }
    r.g = lo;
    const int mt = ts[lo + 1] - ts[lo];
    const int tl = w - ts[lo] * n_tiles;
    r.n_tile = tl / mt;
    r.row0 = offs[lo] + (tl - r.n_tile * mt) * TILE_ROWS + sub;
    r.rows = min(BM, offs[lo + 1] - r.row0);
    return r;
}

struct Piece {
    int tile, kb0, kb1;
};

struct Walk {
    int tile, step, full, k_blocks;
    int64_t pos, end;

    __device__ __forceinline__ Walk(const Plan& p, int unit, int n_units, int k_blocks_)
        : tile(unit), step(n_units), full(p.full), k_blocks(k_blocks_), pos(0), end(0)
    {
        if (unit < p.segments) {
            const int64_t total = (int64_t)(p.tiles - p.full) * k_blocks;
            pos = total * unit / p.segments;
            end = total * (unit + 1) / p.segments;
        }
    }

    __device__ __forceinline__ bool next(Piece& p)
    {
        if (tile < full) {
            p = {tile, 0, k_blocks};
            tile += step;
            return true;
        }
        if (pos >= end) return false;
        const int q = (int)(pos / k_blocks);
        p.tile = full + q;
        p.kb0 = (int)(pos - (int64_t)q * k_blocks);
        p.kb1 = (int)min((int64_t)k_blocks, p.kb0 + (end - pos));
        pos += p.kb1 - p.kb0;
        return true;
    }
};

// The parts of tile q of the segments' tiles: the first segment that holds
// blocks of it, and how many do. Segment c keeps a part that begins with its
// tile in slot 2c + 1, one that begins inside it in slot 2c.
__device__ __forceinline__ int first_part(const Plan& p, int q, int k_blocks, int& parts)
{
    const int64_t total = (int64_t)(p.tiles - p.full) * k_blocks;
    auto segment_of = [&](int64_t block) { return (int)(((block + 1) * p.segments - 1) / total); };
    const int first = segment_of((int64_t)q * k_blocks);
    parts = segment_of((int64_t)(q + 1) * k_blocks - 1) - first + 1;
    return first;
}

// The join of a tile's parts (below): rows of a warp and parts whose loads are in
// flight together. More of either spill the registers of the fold (measured:
// a gated batch 72 -> 107 us).
template <int BN>
constexpr int JOIN_ROWS = BN == 256 ? 2 : 4;
constexpr int JOIN_PARTS = 2;

// The plan with the least estimated time, counted in K blocks of one CTA (0.42
// us), one candidate a lane (the warp calls it together): lane 0 every tile
// whole, which costs its blocks and kFp8TileCost; lane l the tiles, where they
// fill less than one round, in l + 1 parts each; lane 31 the tiles beyond the
// whole rounds but one (or all of them) in equal runs. Cutting costs the parts'
// publication, twice where the runs do not line up with tiles, and the join's
// trips to L2. Measured (us, whole tiles / best cut): one row, 16 tiles of 112
// blocks for each of 2 experts 55.6 / 27.8; 64 rows, 16 tiles of 32 blocks 17.2
// / 15.7; 128 rows, 16 tiles of 32 blocks 19.4 / 22.7; 333 rows, 42 tiles of 160
// blocks 74.7 / 43.
template <int BN>
__device__ __forceinline__ Plan make_plan(int tiles, int rows, int k_blocks, int n_cta, int lane)
{
    // what a tile, a cut and a join cost beside the blocks, in blocks: more of the
    // shorter ones of 128 columns (with 1.3, the blocks' own ratio, 16 rows of K =
    // 2048, N = 4096 take 10.5 us instead of 9.4, 2048 rows of K = 4096, N = 256 17.7
    // instead of 14.9, and 15 other shapes the same)
    constexpr float unit = BN == 256 ? 1.0f : 1.6f;
    constexpr int join_rows = FOLD_WARPS * JOIN_ROWS<BN>;
    const bool room = (int64_t)2 * n_cta * rows <= kFp8PartRows && 2 * n_cta <= kFp8MaxTickets;
    const int rounds = tiles / n_cta;
    const float whole = (float)k_blocks + unit * kFp8TileCost;
    int full = tiles, segments = 0, parts = 0;
    float cost = (float)((tiles + n_cta - 1) / n_cta) * whole;
    bool fits = lane == 0;
    if (lane > 0 && room && tiles > 0) {
        full = rounds > 1 ? (rounds - 1) * n_cta : 0;
        segments = lane == 31 ? n_cta : tiles * (lane + 1);
        parts = lane == 31 ? n_cta / (tiles - full) + 2 : lane + 1;
        const int64_t total = (int64_t)(tiles - full) * k_blocks;
        fits = total >= (int64_t)2 * segments &&
               (lane == 31 ? tiles % n_cta != 0 : lane < kFp8MaxSplit && segments <= n_cta);
        cost = (float)(full / n_cta) * whole + (float)((total + segments - 1) / segments) +
               unit * ((lane == 31 ? 2.0f : 1.0f) * kFp8CutCost +
                       kFp8JoinCost * (float)((rows + join_rows - 1) / join_rows) *
                           (float)((parts + JOIN_PARTS - 1) / JOIN_PARTS));
    }
    // the least cost (its low bits give way to the lane)
    const uint32_t key = fits ? (__float_as_uint(cost) & ~31u) | (uint32_t)lane : 0xffffffffu;
    const int best = (int)(__reduce_min_sync(0xffffffffu, key) & 31u);
    return Plan{tiles, __shfl_sync(0xffffffffu, full, best), __shfl_sync(0xffffffffu, segments, best), rows};
}

__device__ __forceinline__ void fold_barrier()   // the fold warps only
{
    asm volatile("bar.sync 1, %0;" ::"n"(FOLD_THREADS) : "memory");
}

// acc[C .. C + 31] += v[0 .. 31] * f
template <int C, int N>
__device__ __forceinline__ void fold32(float (&acc)[N], const uint32_t (&v)[32], float f)
{
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[C + i] = fmaf(__uint_as_float(v[i]), f, acc[C + i]);
}

// Where row p of a product goes and what it is scaled by: false if nowhere.
__device__ __forceinline__ bool row_target(const Fp8GemmArgs& args, int p, int64_t& row, float& wt)
{
    row = p;
    wt = 1.0f;
    if (args.src_row) {
        // scattered: assignment f = src_row[p] goes to slot[f mod k][f / k]
        const int f = args.src_row[p];
        const int64_t t = f / args.k;
        if (f < 0 || t >= args.T) {
            report_error(args.err, MOE_DEV_ERR_BOUNDS);
            return false;
        }
        row = (int64_t)(f - (int)t * args.k) * args.T + t;
        wt = args.topk_w[f];
    } else if (args.topk_w) {
        wt = args.topk_w[p];
    }
    return true;
}

// Writes 64 bytes of each of this warp's 32 rows (lane l holds row l's in v) to
// out[i] + at, out[i] being row 8 i + l / 4 of lane l (null: not written). A lane's
// own bytes would touch 32 lines with every store; through shared memory (16-byte
// pieces swizzled by the row pair, so neither side has bank conflicts) a store
// covers 8 rows' 64 contiguous bytes.
__device__ __forceinline__ void store_rows(uint4* buf, int lane, const uint4 (&v)[4], unsigned char* const (&out)[4],
                                           int64_t at, bool here)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) buf[lane * 4 + (j ^ ((lane >> 1) & 3))] = v[j];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 2);
        const uint4 o = buf[row * 4 + ((lane & 3) ^ ((row >> 1) & 3))];
        if (here && out[i]) *reinterpret_cast<uint4*>(out[i] + at) = o;
    }
    __syncwarp();
}

// The join of a tile's parts, `stride` floats each, added in the order of their
// blocks, and its epilogue: a warp takes JOIN_ROWS rows at a time, a lane 4
// columns of each half of a row, with JOIN_PARTS parts' loads in flight together
// (the parts were just written, so a load is a trip to L2; what bounds the join
// is the number of trips, not the bytes).
template <bool GATED, typename OUT, int BN>
__device__ __forceinline__ void join(const Fp8GemmArgs& args, const Tile& it, int first, int parts, int stride,
                                     int n_blocks, int warp, int lane)
{
    constexpr int ROWS = JOIN_ROWS<BN>;
    constexpr bool TWO = BN == 256;   // a second 4 columns: of W3, or 128 further on
    // the first part begins with the tile, the others inside it (first_part)
    const float* base = args.part + (int64_t)2 * first * stride;
    auto slot = [&](int s) { return (int64_t)(s == 0 ? 1 : 2 * s) * stride; };
    // gated: 4 columns of W1's sums and the same of W3's, 64 further on
    const int c0 = GATED ? (lane >> 4) * 128 + (lane & 15) * 4 : lane * 4;
    const int c1 = c0 + (GATED ? 64 : 128);
    for (int r0 = warp * ROWS; r0 < it.rows; r0 += FOLD_WARPS * ROWS) {
        float4 a[ROWS], b[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) a[q] = b[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s0 = 0; s0 < parts; s0 += JOIN_PARTS) {
            float4 x[JOIN_PARTS][ROWS], y[JOIN_PARTS][ROWS];
#pragma unroll
            for (int s = 0; s < JOIN_PARTS; ++s)
#pragma unroll
                for (int q = 0; q < ROWS; ++q)
                    if (s0 + s < parts && r0 + q < it.rows) {
                        const float* src = base + slot(s0 + s) + (r0 + q) * BN;
                        x[s][q] = __ldcg(reinterpret_cast<const float4*>(src + c0));
                        if (TWO) y[s][q] = __ldcg(reinterpret_cast<const float4*>(src + c1));
                    }
#pragma unroll
            for (int s = 0; s < JOIN_PARTS; ++s)
#pragma unroll
                for (int q = 0; q < ROWS; ++q)
                    if (s0 + s < parts && r0 + q < it.rows) {
                        a[q].x += x[s][q].x; a[q].y += x[s][q].y; a[q].z += x[s][q].z; a[q].w += x[s][q].w;
                        if (TWO) {
                            b[q].x += y[s][q].x; b[q].y += y[s][q].y; b[q].z += y[s][q].z; b[q].w += y[s][q].w;
                        }
                    }
        }
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            if (r0 + q >= it.rows) break;
            const int p = it.row0 + r0 + q;
            if constexpr (GATED) {
                const float h[4] = {silu(a[q].x) * b[q].x, silu(a[q].y) * b[q].y, silu(a[q].z) * b[q].z,
                                    silu(a[q].w) * b[q].w};
                float amax = max_nan(max_nan(fabsf(h[0]), fabsf(h[1])), max_nan(fabsf(h[2]), fabsf(h[3])));
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                const float scale = fp8_scale(amax);
                const float inv = 1.0f / scale;
                const int n = it.n_tile * 128 + lane * 4;
                if (n < args.N)
                    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(args.out) + (int64_t)p * args.N + n) =
                        e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
                if (lane == 0) args.out_scale[(int64_t)p * n_blocks + it.n_tile] = scale;
            } else {
                int64_t row;
                float wt;
                if (!row_target(args, p, row, wt)) continue;
                OUT* dst = static_cast<OUT*>(args.out) + row * args.N;
                const int n = it.n_tile * BN + lane * 4;
                if (n < args.N) store4(dst + n, a[q].x * wt, a[q].y * wt, a[q].z * wt, a[q].w * wt);
                if (TWO && n + 128 < args.N)
                    store4(dst + n + 128, b[q].x * wt, b[q].y * wt, b[q].z * wt, b[q].w * wt);
            }
        }
    }
}

template <bool GATED, typename OUT, bool PAIR, int BN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                const __grid_constant__ CUtensorMap tmB1, const Fp8GemmArgs args)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t tiles_addr = (raw_addr + 1023u) & ~1023u;
    static_assert(BN == 256 || (!GATED && !PAIR), "128 columns: a product, one CTA per MMA");
    using C = Cfg<PAIR, BN>;
    constexpr int HALF = BN / 2;       // columns of a fold thread
    constexpr int STAGES = C::STAGES;
    constexpr int STAGE_BYTES = C::STAGE_BYTES;
    constexpr int CG = PAIR ? 2 : 1;   // tcgen05 CTA group
    SmemTail<STAGES>* st = reinterpret_cast<SmemTail<STAGES>*>(smem_raw + (tiles_addr - raw_addr) +
                                                               (size_t)STAGES * STAGE_BYTES);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = args.G;
    // a pair walks the schedule together, each CTA with its half of every tile's rows
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const int unit = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int n_units = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    const int sub = (int)rank * BM;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&st->full[s]), 1);
            mbar_init(smem_u32(&st->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&st->tfull[a]), 1 + FACTOR_WARPS);
            mbar_init(smem_u32(&st->tempty[a]), PAIR ? 2 * FOLD_WARPS : FOLD_WARPS);
            mbar_init(smem_u32(&st->ffree[a]), FOLD_WARPS);
        }
        mbar_init(smem_u32(&st->drain), 1);
        st->abort = 0;
        fence_barrier_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB0);
        if (GATED) tma_prefetch_desc(&tmB1);
    }
    if (warp == 9) {
        tmem_alloc<CG>(smem_u32(&st->tmem_base), C::TMEM_COLS);
        tmem_relinquish<CG>();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {
        // the tile table from the group offsets (a scan, 32 groups at a time);
        // offsets that decrease or leave [0, R] are reported and give no tiles
        // at all, so no row outside the operands is touched
        bool good = true;
        int tiles = 0;
        int most = 0;   // rows of the fullest tile
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + lane;
            int n = 0;
            if (g < G) {
                const int first = args.offsets ? args.offsets[g] : 0;
                const int end = args.offsets ? args.offsets[g + 1] : args.R;
                good = good && first >= 0 && first <= end && end <= args.R;
                st->offsets[g] = first;
                if (g == G - 1) st->offsets[G] = end;
                n = good ? (end - first + C::TILE_ROWS - 1) / C::TILE_ROWS : 0;
                most = max(most, min(end - first, BM));
            }
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += v;
            }
            if (g < G) st->tile_start[g] = tiles + incl - n;
            tiles += __shfl_sync(0xffffffffu, incl, 31);
        }
        good = __all_sync(0xffffffffu, good);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            st->tile_start[G] = good ? tiles : 0;
            st->most_rows = most;
            if (!good) report_error(args.err, MOE_DEV_ERR_BOUNDS);
        }
    }
    tc_fence_before();
    // a pair: both CTAs' barriers are initialised before either signals the other's
    if (PAIR) cluster_sync(); else __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = st->tmem_base;
    const int n_out = GATED ? BN / 2 : BN;   // output columns of a tile
    const int n_tiles = (args.N + n_out - 1) / n_out;
    const int k_blocks = (args.K + BK - 1) / BK;
    const int all_tiles = st->tile_start[G] * n_tiles;
    const Plan plan = PAIR ? Plan{all_tiles, all_tiles, 0, 0}   // pairs cut nothing
                           : make_plan<BN>(all_tiles, st->most_rows, k_blocks, n_units, lane);
    volatile int* abort = &st->abort;

    if (warp >= 8) {
        setmaxnreg_dec<OTHER_REGS>();
        if (warp == 8) {
            // ============================ TMA producer ============================
            if (lane == 0) {
                int stage = 0;
                uint32_t phase = 0;
                int issued = 0;
                bool ok = true;
                Walk walk(plan, unit, n_units, k_blocks);
                for (Piece pc; ok && walk.next(pc);) {
                    const Tile it = decode_tile<C::TILE_ROWS>(pc.tile, n_tiles, st->tile_start, st->offsets, G, sub);
                    const int n0 = it.n_tile * n_out;
                    for (int kb = pc.kb0; kb < pc.kb1; ++kb) {
                        if (!mbar_wait(smem_u32(&st->empty[stage]), phase ^ 1u, abort, args.err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t full = smem_u32(&st->full[stage]);
                        const uint32_t a_dst = tiles_addr + stage * STAGE_BYTES;
                        const uint32_t b_dst = a_dst + A_BYTES;
                        if constexpr (PAIR) {
                            // both CTAs' boxes complete on rank 0's barrier, which expects
                            // the bytes of the two; rank 1 stages the last 128 columns' rows
                            if (rank == 0) mbar_arrive_expect_tx(full, 2 * STAGE_BYTES);
                            const uint32_t bar = mapa_shared(full, 0);
                            tma_load_2d_pair(a_dst, &tmA, kb * BK, it.row0, bar);
                            if (GATED) {
                                const int n = n0 + (int)rank * 64;
                                tma_load_3d_pair(b_dst, &tmB0, kb * BK, n, it.g, bar);
                                tma_load_3d_pair(b_dst + 64 * BK, &tmB1, kb * BK, n, it.g, bar);
                            } else {
                                tma_load_3d_pair(b_dst, &tmB0, kb * BK, n0 + (int)rank * 128, it.g, bar);
                            }
                            ++issued;
                            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                            continue;
                        }
                        mbar_arrive_expect_tx(full, STAGE_BYTES);
                        tma_load_2d(a_dst, &tmA, kb * BK, it.row0, full);
                        if (GATED) {
                            // columns 0..127 of the MMA: W1 and W3 of the slice's first 64
                            // columns; 128..255: of its last 64 (one half per fold group)
                            tma_load_3d(b_dst, &tmB0, kb * BK, n0, it.g, full);
                            tma_load_3d(b_dst + 64 * BK, &tmB1, kb * BK, n0, it.g, full);
                            tma_load_3d(b_dst + 128 * BK, &tmB0, kb * BK, n0 + 64, it.g, full);
                            tma_load_3d(b_dst + 192 * BK, &tmB1, kb * BK, n0 + 64, it.g, full);
                        } else {
                            tma_load_3d(b_dst, &tmB0, kb * BK, n0, it.g, full);
                        }
                        ++issued;
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    }
                }
                if (!PAIR && !ok) {
                    // drain: wait (bounded) for the loads still in flight
                    for (int i = 0; i < min(issued, STAGES); ++i) {
                        if (stage == 0) { stage = STAGES - 1; phase ^= 1u; } else { --stage; }
                        mbar_wait_drain(smem_u32(&st->full[stage]), phase);
                    }
                }
            }
            __syncwarp();
        } else if (warp == 9) {
            // ============================ MMA issuer ==============================
            // the whole warp walks the pieces and waits (uniform control flow, so the
            // descriptors stay in uniform registers); one elected lane issues (a
            // pair: of the rank-0 CTA, for both)
            const uint32_t leader = elect_one_sync();
            const uint64_t a_desc = smem_desc_sw128(tiles_addr, 16, 1024);
            const uint64_t b_desc = smem_desc_sw128(tiles_addr + A_BYTES, 16, 1024);
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            bool any = false;
            Walk walk(plan, unit, n_units, k_blocks);
            for (Piece pc; ok && rank == 0 && walk.next(pc);) {
                for (int kb = pc.kb0; kb < pc.kb1; ++kb) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(smem_u32(&st->full[stage]), phase, abort, args.err) &&
                                        mbar_wait<PAIR, PAIR>(smem_u32(&st->tempty[acc]), acc_phase ^ 1u, abort, args.err));
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t d = tmem_base + acc * BN;
                        const uint64_t at = (uint64_t)(stage * (STAGE_BYTES >> 4));
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk)
                            // K-major A and B: each K step of 32 is 32 bytes further along the row
                            tc_mma_f8<CG>(d, a_desc + at + 2 * kk, b_desc + at + 2 * kk, C::IDESC, kk != 0 ? 1u : 0u);
                        // one commit for the block: the fold warps give the stage back
                        tc_commit<CG>(smem_u32(&st->tfull[acc]));
                    }
                    __syncwarp();
                    any = true;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
                }
            }
            if (!ok && any && leader) {
                // drain: every MMA issued so far must finish before TMEM is freed
                if (PAIR) tc_commit_pair_local(smem_u32(&st->drain));
                else tc_commit(smem_u32(&st->drain));
                mbar_wait_drain(smem_u32(&st->drain), 0);
            }
            __syncwarp();
        } else {
            // =========================== block factors ============================
            // sa * sw of every row of the tile, for each block: 64 rows a warp, two a
            // lane, written beside the block's sums (tfull counts both)
            const int n_blocks = (args.N + kFp8Block - 1) / kFp8Block;
            const int r0 = (warp - 10) * 64 + lane;
            int buf = 0;
            uint32_t buf_phase = 0;
            bool ok = true;
            Walk walk(plan, unit, n_units, k_blocks);
            Piece pc;
            bool have = walk.next(pc);
            int n = 0, kb = 0;
            const float *sa0 = nullptr, *sa1 = nullptr, *sw0 = nullptr, *sw1 = nullptr;
            Tile it;
            auto enter = [&]() {   // the piece's scales
                it = decode_tile<C::TILE_ROWS>(pc.tile, n_tiles, st->tile_start, st->offsets, G, sub);
                kb = pc.kb0;
                sa0 = args.a_scale + (int64_t)min(it.row0 + r0, args.R - 1) * k_blocks;
                sa1 = args.a_scale + (int64_t)min(it.row0 + r0 + 32, args.R - 1) * k_blocks;
                // gated: the slice's block of W1 and of W3; product: each half's block
                const int64_t b0 = (int64_t)it.g * n_blocks + (GATED || BN == 128 ? it.n_tile : 2 * it.n_tile);
                const int64_t b1 = GATED || BN == 128 || 2 * it.n_tile + 1 == n_blocks ? b0 : b0 + 1;
                sw0 = args.w0_scale + b0 * k_blocks;
                sw1 = (GATED ? args.w1_scale : args.w0_scale) + b1 * k_blocks;
            };
            float x0 = 0.0f, x1 = 0.0f, y0 = 0.0f, y1 = 0.0f;
            auto fetch = [&]() {
                x0 = __ldg(sa0 + kb);
                x1 = __ldg(sa1 + kb);
                y0 = __ldg(sw0 + kb);
                y1 = __ldg(sw1 + kb);
            };
            if (have) {
                enter();
                fetch();
            }
            while (have) {
                const float2 f0 = make_float2(x0 * y0, x0 * y1), f1 = make_float2(x1 * y0, x1 * y1);
                const bool opens = kb == pc.kb0;
                const Tile now = it;
                const int slot = n % TILE_SLOTS;
                // the next block's scales, of the next piece after the last, while the
                // slot is waited for
                if (++kb == pc.kb1) {
                    have = walk.next(pc);
                    ++n;
                    if (have) enter();
                }
                if (have) fetch();
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&st->ffree[buf]), buf_phase ^ 1u, abort, args.err));
                if (!ok) break;
                if (opens && warp == 10 && lane == 0) st->tile[slot] = now;
                st->factor[buf][r0] = f0;
                st->factor[buf][r0 + 32] = f1;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&st->tfull[buf]));
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            }
        }
    } else {
        setmaxnreg_inc<FOLD_REGS>();
        // ========================= fold and epilogue ==========================
        const int half = warp >> 2;                  // MMA columns HALF half .. + HALF - 1
        const int r = (warp & 3) * 32 + lane;        // row of the tile = TMEM lane
        const uint32_t t_row = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + half * HALF;
        int stage = 0;
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ready = false;    // the next block is known to be there
        // after an abort every fold warp still walks all pieces, without waiting
        // for the tensor cores, so that the barriers below stay matched
        bool ok = true;
        Walk walk(plan, unit, n_units, k_blocks);
        int n = 0;
        for (Piece pc; walk.next(pc); ++n) {
            float acc[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) acc[i] = 0.0f;
            for (int kb = pc.kb0; kb < pc.kb1 && ok; ++kb) {
                ok = __all_sync(0xffffffffu, ready || mbar_wait(smem_u32(&st->tfull[buf]), buf_phase, abort, args.err));
                if (!ok) break;
                tc_fence_after();
                const uint32_t t = t_row + buf * BN;
                // the block's MMAs are done, so its stage may be loaded again
                if (threadIdx.x == 0) mbar_arrive(smem_u32(&st->empty[stage]));
                if (++stage == STAGES) stage = 0;
                const float2 f = st->factor[buf][r];
                const float c0 = GATED || half == 0 ? f.x : f.y;
                const float c1 = GATED ? f.y : c0;
                uint32_t u[32], v[32];
                tmem_ld_32x32b_x32(t, u);
                tmem_ld_32x32b_x32(t + 32, v);
                tc_wait_ld_for(u);
                tc_wait_ld_for(v);
                if constexpr (HALF == 128) {
                    fold32<0>(acc, u, c0);
                    tmem_ld_32x32b_x32(t + 64, u);
                    fold32<32>(acc, v, c0);
                    tmem_ld_32x32b_x32(t + 96, v);
                    tc_wait_ld_for(u);
                    tc_wait_ld_for(v);
                }
                // TMEM is read: the tensor cores may fill this buffer again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&st->ffree[buf]));
                    if (PAIR && rank != 0) mbar_arrive_remote_tmem(mapa_shared(smem_u32(&st->tempty[buf]), 0));
                    else mbar_arrive(smem_u32(&st->tempty[buf]));
                }
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
                // whether the next block is there, asked before this one's last sums
                ready = mbar_test(smem_u32(&st->tfull[buf]), buf_phase);
                if constexpr (HALF == 128) {
                    fold32<64>(acc, u, c1);
                    fold32<96>(acc, v, c1);
                } else {
                    fold32<0>(acc, u, c0);
                    fold32<32>(acc, v, c0);
                }
            }

            const int n_blocks = (args.N + kFp8Block - 1) / kFp8Block;
            const Tile it = ok ? st->tile[n % TILE_SLOTS] : Tile{0, 0, 0, 0};
            const bool valid = r < it.rows;
            const int p = it.row0 + r;
            if (pc.kb1 - pc.kb0 < k_blocks) {
                // publish this piece's part (its rows side by side) and take a ticket;
                // the last piece of the tile joins the parts
                float* part = args.part + ((int64_t)(2 * unit + (pc.kb0 == 0)) * plan.part_rows + r) * BN + half * HALF;
                if (ok && valid) {
#pragma unroll
                    for (int c = 0; c < HALF; c += 8)
                        st_global_v8(part + c, __float_as_uint(acc[c]), __float_as_uint(acc[c + 1]),
                                     __float_as_uint(acc[c + 2]), __float_as_uint(acc[c + 3]),
                                     __float_as_uint(acc[c + 4]), __float_as_uint(acc[c + 5]),
                                     __float_as_uint(acc[c + 6]), __float_as_uint(acc[c + 7]));
                }
                __threadfence();
                fold_barrier();
                const int q = pc.tile - plan.full;
                int parts;
                const int first = first_part(plan, q, k_blocks, parts);
                if (threadIdx.x == 0) {
                    int last = 0;
                    if (!*abort) {
                        last = atomicAdd(args.ticket + q, 1) == parts - 1;
                        if (last) args.ticket[q] = 0;   // as found, for the next call
                    }
                    __threadfence();
                    st->last = last;
                }
                fold_barrier();
                if (st->last)
                    join<GATED, OUT, BN>(args, it, first, parts, plan.part_rows * BN, n_blocks, warp, lane);
                continue;
            }

            if constexpr (GATED) {
                // h = silu(a W1^T) * (a W3^T) of this thread's row and 64 columns
                const int n0 = it.n_tile * 128 + half * 64;
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    acc[i] = silu(acc[i]) * acc[64 + i];
                    // columns past N are zero (zero weights): they do not count
                    amax = max_nan(amax, fabsf(acc[i]));
                }
                // the block's maximum: this half's and the other's
                st->amax[n & 1][half][r] = amax;
                fold_barrier();
                amax = max_nan(amax, st->amax[n & 1][half ^ 1][r]);
                const float scale = fp8_scale(amax);
                const float inv = 1.0f / scale;
                unsigned char* out[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = (warp & 3) * 32 + 8 * i + (lane >> 2);
                    out[i] = ok && row < it.rows
                                 ? static_cast<unsigned char*>(args.out) + (int64_t)(it.row0 + row) * args.N + n0
                                 : nullptr;
                }
                uint4 o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float* h = acc + 16 * i;
                    o[i].x = e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
                    o[i].y = e4m3x4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv);
                    o[i].z = e4m3x4(h[8] * inv, h[9] * inv, h[10] * inv, h[11] * inv);
                    o[i].w = e4m3x4(h[12] * inv, h[13] * inv, h[14] * inv, h[15] * inv);
                }
                store_rows(st->stage_out[warp], lane, o, out, (lane & 3) * 16, n0 + (lane & 3) * 16 < args.N);
                if (valid && ok && half == 0) args.out_scale[(int64_t)p * n_blocks + it.n_tile] = scale;
            } else {
                const int n0 = it.n_tile * BN + half * HALF;
                int64_t row = 0;
                float wt = 1.0f;
                const bool mine = ok && valid && row_target(args, p, row, wt);
                const unsigned there = __ballot_sync(0xffffffffu, mine);
                unsigned char* out[4];   // of the rows that this lane stores (store_rows)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int l = 8 * i + (lane >> 2);
                    const int64_t at = __shfl_sync(0xffffffffu, row, l);
                    out[i] = (there >> l) & 1
                                 ? reinterpret_cast<unsigned char*>(static_cast<OUT*>(args.out) + at * args.N + n0)
                                 : nullptr;
                }
                constexpr int COLS = 64 / (int)sizeof(OUT);   // columns of a row at once
                constexpr int PIECE = 16 / (int)sizeof(OUT);  // and of a 16-byte piece
#pragma unroll
                for (int c = 0; c < HALF; c += COLS) {
                    uint4 o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float* q = acc + c + PIECE * j;
                        if constexpr (sizeof(OUT) == 2)
                            o[j] = make_uint4(bf16x2(q[0] * wt, q[1] * wt), bf16x2(q[2] * wt, q[3] * wt),
                                              bf16x2(q[4] * wt, q[5] * wt), bf16x2(q[6] * wt, q[7] * wt));
                        else
                            o[j] = make_uint4(__float_as_uint(q[0] * wt), __float_as_uint(q[1] * wt),
                                              __float_as_uint(q[2] * wt), __float_as_uint(q[3] * wt));
                    }
                    const int n = c + (lane & 3) * PIECE;
                    store_rows(st->stage_out[warp], lane, o, out, (int64_t)n * (int)sizeof(OUT), n0 + n < args.N);
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
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc<CG>(tmem_base, C::TMEM_COLS);
    }
}

constexpr int kMaxDevices = 64;

// Lets `kern` have `bytes` of dynamic shared memory on the current device, asked
// of the runtime once per kernel (its bit set in `done`) and device.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, std::atomic<uint64_t>& done, int& dev)
{
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const uint64_t bit = (uint64_t)1 << dev;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// CTA-pair kernels: how many pairs can be resident at once (shared memory and
// the GPCs' SM pairs decide), looked up once per kernel and device.
std::atomic<int> g_pairs[3][kMaxDevices];

template <bool GATED, typename OUT>
cudaError_t launch_pair(int slot, const CUtensorMap& tmA, const CUtensorMap& tmB0, const CUtensorMap& tmB1,
                        const Fp8GemmArgs& a, int num_sms, cudaStream_t s)
{
    auto kern = fp8_gemm_kernel<GATED, OUT, true, 256>;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = allow_smem(kern, smem_bytes<true, 256>(), done, dev);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = smem_bytes<true, 256>();
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int pairs = g_pairs[slot][dev].load(std::memory_order_relaxed);
    if (pairs <= 0) {
        cfg.gridDim = dim3((unsigned)(num_sms & ~1));
        e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
        if (e != cudaSuccess) return e;
        if (pairs <= 0) return cudaErrorInvalidConfiguration;
        g_pairs[slot][dev].store(pairs, std::memory_order_relaxed);
    }
    pairs = pairs < num_sms / 2 ? pairs : num_sms / 2;
    if (pairs <= 0) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.numAttrs = 2;   // the cached occupancy query above saw the cluster shape only
    e = cudaLaunchKernelEx(&cfg, kern, tmA, tmB0, tmB1, a);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <bool GATED, typename OUT, int BN>
cudaError_t launch(const CUtensorMap& tmA, const CUtensorMap& tmB0, const CUtensorMap& tmB1, const Fp8GemmArgs& a,
                   int num_sms, cudaStream_t s)
{
    auto kern = fp8_gemm_kernel<GATED, OUT, false, BN>;
    constexpr size_t smem = smem_bytes<false, BN>();
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    const cudaError_t e = allow_smem(kern, smem, done, dev);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(num_sms), dim3(NUM_THREADS), smem, s, tmA, tmB0, tmB1, a);
}

template <typename OUT>
cudaError_t launch_product(Fp8GemmForm form, int slot, const CUtensorMap& tmA, const CUtensorMap& tmB,
                           const Fp8GemmArgs& a, int num_sms, cudaStream_t s)
{
    if (form == kFp8Pair) return launch_pair<false, OUT>(slot, tmA, tmB, tmB, a, num_sms, s);
    if (form == kFp8Narrow) return launch<false, OUT, 128>(tmA, tmB, tmB, a, num_sms, s);
    return launch<false, OUT, 256>(tmA, tmB, tmB, a, num_sms, s);
}

}  // namespace

cudaError_t launch_fp8_gemm(Fp8GemmMode mode, Fp8GemmForm form, const CUtensorMap& tmA, const CUtensorMap& tmB0,
                            const CUtensorMap& tmB1, const Fp8GemmArgs& a, int num_sms, cudaStream_t s)
{
    if (a.R == 0) return cudaSuccess;
    if (a.R < 0 || a.G < 1 || a.G > MAX_GROUPS || (!a.offsets && a.G != 1)) return cudaErrorInvalidValue;
    switch (mode) {
    case kFp8Gated:
        if (form == kFp8Narrow) return cudaErrorInvalidValue;
        return form == kFp8Pair ? launch_pair<true, uint8_t>(0, tmA, tmB0, tmB1, a, num_sms, s)
                                : launch<true, uint8_t, 256>(tmA, tmB0, tmB1, a, num_sms, s);
    case kFp8ProductBf16: return launch_product<__nv_bfloat16>(form, 1, tmA, tmB0, a, num_sms, s);
    case kFp8ProductF32: return launch_product<float>(form, 2, tmA, tmB0, a, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
