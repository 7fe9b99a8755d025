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
// of (expert, N tile, M tile, K split) items computed from the group offsets:
//   warps 0..7  fold and epilogue: warp w reads TMEM lanes 32 (w mod 4) .. + 31
//               (rows) and columns 128 (w / 4) .. + 127: 128 fp32 accumulators a
//               thread;
//   warp 8      TMA producer: 4-stage ring of {A 128 x 128, B 256 x 128} bytes;
//   warp 9      TMEM allocator and MMA issuer;
//   warps 10,11 the rows' factors sa * sw of each block, into shared memory.
// CTA pairs (PAIR): a 2-CTA cluster shares one tcgen05.mma.cta_group::2 of M =
// 256; both CTAs' boxes complete on rank 0's barrier, rank 0 issues, its commit
// arrives in both CTAs, and both CTAs' fold warps release a buffer on rank 0.
// When there are too few tiles for the SMs (few rows), K is split over several
// items of one tile; each writes its fp32 partial sums to the workspace, takes
// a ticket, and the last one adds the parts in split order (so the result does
// not depend on which came last) and runs the epilogue. No CTA waits for
// another. Every wait is bounded (ptx.cuh).
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
constexpr int BN = 256;            // MMA N (gated: 128 of W1 and 128 of W3, interleaved by 64)
constexpr int BK = kFp8Block;      // one scale block of K = one 128-byte swizzle span
constexpr int A_BYTES = BM * BK;   // 16 KB
constexpr int FOLD_WARPS = 8;
constexpr int FOLD_THREADS = 32 * FOLD_WARPS;
constexpr int FACTOR_WARPS = 2;
constexpr int NUM_THREADS = FOLD_THREADS + 128;
// registers: 12 warps are launched with 168 each; the fold warps (128
// accumulators, two 32-column loads in flight) take 216 once the other
// warpgroup has gone down to 72 (8 * 216 + 4 * 72 = 12 * 168)
constexpr int FOLD_REGS = 216;
constexpr int OTHER_REGS = 72;
constexpr int MAX_GROUPS = 256;
constexpr int TMEM_COLS = 512;

// One CTA per MMA (PAIR false): a stage holds 128 rows of A and 256 of B. A CTA
// pair (tcgen05 cta_group::2): one MMA of 256 x 256 over both CTAs, each staging
// its 128 rows of A and half of B's, so a third less comes from L2 per block.
template <bool PAIR>
struct Cfg {
    static constexpr int B_ROWS = PAIR ? BN / 2 : BN;
    static constexpr int STAGE_BYTES = A_BYTES + B_ROWS * BK;   // 48 KB or 32 KB
    static constexpr int STAGES = PAIR ? 6 : 4;
    static constexpr int TILE_ROWS = PAIR ? 2 * BM : BM;        // rows of one work item
    static constexpr uint32_t IDESC = idesc_e4m3_f32(TILE_ROWS, BN);
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
    int last;                          // K split: this item took its tile's last ticket
    int tile_start[MAX_GROUPS + 1];    // tiles before each group
    int offsets[MAX_GROUPS + 1];
    float2 factor[2][BM];              // sa * sw of each row: column halves (gated: W1 and W3)
    float amax[2][2][BM];              // gated: [tile parity][column half][row]
};
template <bool PAIR>
constexpr size_t smem_bytes()
{
    return 1024 + (size_t)Cfg<PAIR>::STAGES * Cfg<PAIR>::STAGE_BYTES + sizeof(SmemTail<Cfg<PAIR>::STAGES>);
}
static_assert(smem_bytes<false>() <= 227 * 1024 && smem_bytes<true>() <= 227 * 1024, "shared memory");

struct Item {
    int g, row0, rows, n_tile, tile, split;
};

// Item w: tile w / S, split w mod S; tiles expert-major, then N tile, then M
// tile (neighbouring CTAs share the weights of an N tile in L2). This CTA's rows
// start `sub` rows into the tile (a pair's rank 1: 128) and may be none (rows <= 0).
template <int TILE_ROWS>
__device__ __forceinline__ Item decode_item(int w, int S, int n_tiles, const int* ts, const int* offs, int G, int sub)
{
    Item r;
    r.tile = w / S;
    r.split = w - r.tile * S;
    int lo = 0, hi = G;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ts[mid] * n_tiles <= r.tile) lo = mid; else hi = mid;
    }
    r.g = lo;
    const int mt = ts[lo + 1] - ts[lo];
    const int tl = r.tile - ts[lo] * n_tiles;
    r.n_tile = tl / mt;
    r.row0 = offs[lo] + (tl - r.n_tile * mt) * TILE_ROWS + sub;
    r.rows = min(BM, offs[lo + 1] - r.row0);
    return r;
}

// How many ways to split K: the S that minimises (rounds of items over the
// CTAs) x (K blocks per item + a fixed cost per item, larger when parts have
// to be joined), with the parts of all items within the workspace.
__device__ __forceinline__ int choose_split(int tiles, int k_blocks, int n_cta)
{
    int best = 1;
    int best_cost = ((tiles + n_cta - 1) / n_cta) * (k_blocks + kFp8ItemCost);
    for (int s = 2; s <= kFp8MaxSplit; ++s) {
        if (tiles * s > kFp8MaxItems || k_blocks < 2 * s) break;
        const int cost = ((tiles * s + n_cta - 1) / n_cta) * ((k_blocks + s - 1) / s + kFp8ItemCost + kFp8JoinCost);
        if (cost < best_cost) {
            best_cost = cost;
            best = s;
        }
    }
    return best;
}

__device__ __forceinline__ void fold_barrier()   // the fold warps only
{
    asm volatile("bar.sync 1, %0;" ::"n"(FOLD_THREADS) : "memory");
}

// acc[C .. C + 31] += v[0 .. 31] * f
template <int C>
__device__ __forceinline__ void fold32(float (&acc)[128], const uint32_t (&v)[32], float f)
{
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[C + i] = fmaf(__uint_as_float(v[i]), f, acc[C + i]);
}

template <bool GATED, typename OUT, bool PAIR>
__global__ void __launch_bounds__(NUM_THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                const __grid_constant__ CUtensorMap tmB1, const Fp8GemmArgs args)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t tiles_addr = (raw_addr + 1023u) & ~1023u;
    using C = Cfg<PAIR>;
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
        tmem_alloc<CG>(smem_u32(&st->tmem_base), TMEM_COLS);
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
        if (lane == 0) {
            st->tile_start[G] = good ? tiles : 0;
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
    const int tiles = st->tile_start[G] * n_tiles;
    const int S = PAIR ? 1 : choose_split(tiles, k_blocks, n_units);
    const int items = tiles * S;
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
                for (int w = unit; w < items && ok; w += n_units) {
                    const Item it = decode_item<C::TILE_ROWS>(w, S, n_tiles, st->tile_start, st->offsets, G, sub);
                    const int kb1 = (it.split + 1) * k_blocks / S;
                    const int n0 = it.n_tile * n_out;
                    for (int kb = it.split * k_blocks / S; kb < kb1; ++kb) {
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
            // the whole warp walks the items and waits (uniform control flow, so the
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
            for (int w = unit; w < items && ok && rank == 0; w += n_units) {
                const int split = w % S;
                const int n_kb = (split + 1) * k_blocks / S - split * k_blocks / S;
                for (int i = 0; i < n_kb; ++i) {
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(smem_u32(&st->full[stage]), phase, abort, args.err) &&
                                        mbar_wait(smem_u32(&st->tempty[acc]), acc_phase ^ 1u, abort, args.err));
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
            for (int w = unit; w < items && ok; w += n_units) {
                const Item it = decode_item<C::TILE_ROWS>(w, S, n_tiles, st->tile_start, st->offsets, G, sub);
                const int kb0 = it.split * k_blocks / S, kb1 = (it.split + 1) * k_blocks / S;
                const float* sa0 = args.a_scale + (int64_t)min(it.row0 + r0, args.R - 1) * k_blocks;
                const float* sa1 = args.a_scale + (int64_t)min(it.row0 + r0 + 32, args.R - 1) * k_blocks;
                // gated: the slice's block of W1 and of W3; product: each half's block
                const int64_t b0 = (int64_t)it.g * n_blocks + (GATED ? it.n_tile : 2 * it.n_tile);
                const int64_t b1 = GATED || 2 * it.n_tile + 1 == n_blocks ? b0 : b0 + 1;
                const float* sw0 = args.w0_scale + b0 * k_blocks;
                const float* sw1 = (GATED ? args.w1_scale : args.w0_scale) + b1 * k_blocks;
                float x0 = __ldg(sa0 + kb0), x1 = __ldg(sa1 + kb0), y0 = __ldg(sw0 + kb0), y1 = __ldg(sw1 + kb0);
                for (int kb = kb0; kb < kb1; ++kb) {
                    const float2 f0 = make_float2(x0 * y0, x0 * y1), f1 = make_float2(x1 * y0, x1 * y1);
                    if (kb + 1 < kb1) {   // the next block's scales, while the slot is waited for
                        x0 = __ldg(sa0 + kb + 1);
                        x1 = __ldg(sa1 + kb + 1);
                        y0 = __ldg(sw0 + kb + 1);
                        y1 = __ldg(sw1 + kb + 1);
                    }
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(smem_u32(&st->ffree[buf]), buf_phase ^ 1u, abort, args.err));
                    if (!ok) break;
                    st->factor[buf][r0] = f0;
                    st->factor[buf][r0 + 32] = f1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&st->tfull[buf]));
                    if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
                }
            }
        }
    } else {
        setmaxnreg_inc<FOLD_REGS>();
        // ========================= fold and epilogue ==========================
        const int half = warp >> 2;                  // MMA columns 128 half .. + 127
        const int r = (warp & 3) * 32 + lane;        // row of the tile = TMEM lane
        const uint32_t t_row = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + half * 128;
        const int n_blocks = (args.N + kFp8Block - 1) / kFp8Block;
        int stage = 0;
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ready = false;    // the next block is known to be there
        uint32_t parity = 0;   // which amax buffer this tile uses
        // after an abort every fold warp still walks all items, without waiting
        // for the tensor cores, so that the barriers below stay matched
        bool ok = true;
        for (int w = unit; w < items; w += n_units) {
            const Item it = decode_item<C::TILE_ROWS>(w, S, n_tiles, st->tile_start, st->offsets, G, sub);
            const bool valid = r < it.rows;
            const int p = it.row0 + r;
            const int kb0 = it.split * k_blocks / S, kb1 = (it.split + 1) * k_blocks / S;
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
            for (int kb = kb0; kb < kb1 && ok; ++kb) {
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
                fold32<0>(acc, u, c0);
                tmem_ld_32x32b_x32(t + 64, u);
                fold32<32>(acc, v, c0);
                tmem_ld_32x32b_x32(t + 96, v);
                tc_wait_ld_for(u);
                tc_wait_ld_for(v);
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
                fold32<64>(acc, u, c1);
                fold32<96>(acc, v, c1);
            }

            if (S > 1) {
                // publish this item's part (columns in fours, rows side by side), take
                // a ticket; the last item of the tile adds the parts in split order
                float4* part = args.part + (int64_t)w * (BM * BN / 4) + (half * 32) * BM + r;
                if (ok && valid) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        __stcg(part + c * BM,
                               make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]));
                    }
                }
                __threadfence();
                fold_barrier();
                if (threadIdx.x == 0) {
                    int last = 0;
                    if (!*abort) {
                        last = atomicAdd(args.ticket + it.tile, 1) == S - 1;
                        if (last) args.ticket[it.tile] = 0;   // as found, for the next call
                    }
                    __threadfence();
                    st->last = last;
                }
                fold_barrier();
                if (!st->last) continue;
                if (valid) {
                    const float4* first = args.part + (int64_t)it.tile * S * (BM * BN / 4) + (half * 32) * BM + r;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float4 sum = __ldcg(first + c * BM);
                        for (int s = 1; s < S; ++s) {
                            const float4 v = __ldcg(first + (int64_t)s * (BM * BN / 4) + c * BM);
                            sum.x += v.x;
                            sum.y += v.y;
                            sum.z += v.z;
                            sum.w += v.w;
                        }
                        acc[4 * c] = sum.x;
                        acc[4 * c + 1] = sum.y;
                        acc[4 * c + 2] = sum.z;
                        acc[4 * c + 3] = sum.w;
                    }
                }
            }

            if constexpr (GATED) {
                // h = silu(a W1^T) * (a W3^T) of this thread's row and 64 columns
                const int n0 = it.n_tile * 128 + half * 64;
                float h[64];
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    h[i] = silu(acc[i]) * acc[64 + i];
                    // columns past N are zero (zero weights): they do not count
                    amax = max_nan(amax, fabsf(h[i]));
                }
                // the block's maximum: this half's and the other's
                st->amax[parity][half][r] = amax;
                fold_barrier();
                amax = max_nan(amax, st->amax[parity][half ^ 1][r]);
                parity ^= 1u;
                const float scale = fp8_scale(amax);
                const float inv = 1.0f / scale;
                if (valid && ok) {
                    uint8_t* dst = static_cast<uint8_t*>(args.out) + (int64_t)p * args.N + n0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (n0 + 16 * i < args.N) {
                            uint4 o;
                            o.x = e4m3x4(h[16 * i] * inv, h[16 * i + 1] * inv, h[16 * i + 2] * inv, h[16 * i + 3] * inv);
                            o.y = e4m3x4(h[16 * i + 4] * inv, h[16 * i + 5] * inv, h[16 * i + 6] * inv, h[16 * i + 7] * inv);
                            o.z = e4m3x4(h[16 * i + 8] * inv, h[16 * i + 9] * inv, h[16 * i + 10] * inv, h[16 * i + 11] * inv);
                            o.w = e4m3x4(h[16 * i + 12] * inv, h[16 * i + 13] * inv, h[16 * i + 14] * inv, h[16 * i + 15] * inv);
                            *reinterpret_cast<uint4*>(dst + 16 * i) = o;
                        }
                    }
                    if (half == 0) args.out_scale[(int64_t)p * n_blocks + it.n_tile] = scale;
                }
            } else if (valid && ok) {
                const int n0 = it.n_tile * BN + half * 128;
                int64_t row = p;
                float wt = 1.0f;
                bool in_bounds = true;
                if (args.src_row) {
                    // scattered: assignment f = src_row[p] goes to slot[f mod k][f / k]
                    const int f = args.src_row[p];
                    const int64_t t = f / args.k;
                    in_bounds = f >= 0 && t < args.T;
                    row = in_bounds ? (int64_t)(f - (int)t * args.k) * args.T + t : 0;
                    if (in_bounds) wt = args.topk_w[f];
                    else report_error(args.err, MOE_DEV_ERR_BOUNDS);
                } else if (args.topk_w) {
                    wt = args.topk_w[p];
                }
                OUT* dst = static_cast<OUT*>(args.out) + row * args.N + n0;
                if (in_bounds) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (n0 + 8 * i < args.N) {
                            float o[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) o[u] = acc[8 * i + u] * wt;
                            store8(dst + 8 * i, o);
                        }
                    }
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
        tmem_dealloc<CG>(tmem_base, TMEM_COLS);
    }
}

// CTA-pair kernels: how many pairs can be resident at once (shared memory and
// the GPCs' SM pairs decide), looked up once per kernel and device.
constexpr int kMaxPairDevices = 64;
std::atomic<int> g_pairs[3][kMaxPairDevices];

template <bool GATED, typename OUT>
cudaError_t launch_pair(int slot, const CUtensorMap& tmA, const CUtensorMap& tmB0, const CUtensorMap& tmB1,
                        const Fp8GemmArgs& a, int num_sms, cudaStream_t s)
{
    auto kern = fp8_gemm_kernel<GATED, OUT, true>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<true>());
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
    cfg.dynamicSmemBytes = smem_bytes<true>();
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxPairDevices) return cudaErrorInvalidDevice;
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

template <bool GATED, typename OUT>
cudaError_t launch(const CUtensorMap& tmA, const CUtensorMap& tmB0, const CUtensorMap& tmB1, const Fp8GemmArgs& a,
                   int num_sms, cudaStream_t s)
{
    auto kern = fp8_gemm_kernel<GATED, OUT, false>;
    constexpr size_t smem = smem_bytes<false>();
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(num_sms), dim3(NUM_THREADS), smem, s, tmA, tmB0, tmB1, a);
}

}  // namespace

cudaError_t launch_fp8_gemm(Fp8GemmMode mode, bool pair, const CUtensorMap& tmA, const CUtensorMap& tmB0,
                            const CUtensorMap& tmB1, const Fp8GemmArgs& a, int num_sms, cudaStream_t s)
{
    if (a.R == 0) return cudaSuccess;
    if (a.R < 0 || a.G < 1 || a.G > MAX_GROUPS || (!a.offsets && a.G != 1)) return cudaErrorInvalidValue;
    switch (mode) {
    case kFp8Gated:
        return pair ? launch_pair<true, uint8_t>(0, tmA, tmB0, tmB1, a, num_sms, s)
                    : launch<true, uint8_t>(tmA, tmB0, tmB1, a, num_sms, s);
    case kFp8ProductBf16:
        return pair ? launch_pair<false, __nv_bfloat16>(1, tmA, tmB0, tmB1, a, num_sms, s)
                    : launch<false, __nv_bfloat16>(tmA, tmB0, tmB1, a, num_sms, s);
    case kFp8ProductF32:
        return pair ? launch_pair<false, float>(2, tmA, tmB0, tmB1, a, num_sms, s)
                    : launch<false, float>(tmA, tmB0, tmB1, a, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
