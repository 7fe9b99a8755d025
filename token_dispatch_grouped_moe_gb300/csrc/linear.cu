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
// The tensor cores' running sum is cut every 512 k: the epilogue warps add each
// stretch to fp32 registers while the next one is computed into the other TMEM
// buffer (its 32 partial sums rounded towards zero are far below a bf16 step; of
// thousands they would not be below fp32's).
//
// Kernel shape: one CTA per SM (384 threads), persistent over (group, row tile, n
// tile) tiles computed from the group offsets:
//   warps 0..7  epilogue: warp w reads TMEM lanes 32 (w mod 4) .. + 31 (columns n,
//               one a thread) and half of the rows;
//   warp 8      TMA producer; warp 9 TMEM allocator and MMA issuer.
// Every wait is bounded (ptx.cuh).
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.cuh"
#include "ops.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int BM = 128;             // columns of the output in a tile
constexpr int BK = kLinearBK;
constexpr int W_BYTES = BM * BK * 2;
constexpr int STRETCH = 8;          // k blocks between two reads of TMEM
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 32 * EPI_WARPS + 128;
// registers: 12 warps are launched with 168 each; the epilogue warps (up to 128
// sums and 64 loads in flight) take 216 once the other warpgroup has gone down to
// 72 (8 * 216 + 4 * 72 = 12 * 168)
constexpr int EPI_REGS = 216;
constexpr int OTHER_REGS = 72;
constexpr int MAX_GROUPS = 256;
constexpr int ROW_STEP = 16;        // the MMA's N is a multiple of this
constexpr int BAND = 16;            // row tiles that are taken together

template <int BN>
struct Cfg {
    static constexpr int STAGE_BYTES = W_BYTES + BN * BK * 2;
    static constexpr int STAGES = BN == 256 ? 4 : 6;
    static constexpr int TMEM_COLS = 2 * BN;
};

struct Tile {
    int g, row0, rows, n0;
};

template <int STAGES>
struct SmemTail {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int tile_start[MAX_GROUPS + 1];    // row tiles before each group
    int offsets[MAX_GROUPS + 1];
};

template <int BN>
constexpr size_t smem_bytes()
{
    return 1024 + (size_t)Cfg<BN>::STAGES * Cfg<BN>::STAGE_BYTES + sizeof(SmemTail<Cfg<BN>::STAGES>);
}
static_assert(smem_bytes<256>() <= 227 * 1024 && smem_bytes<128>() <= 227 * 1024, "shared memory");

// Tile w: group-major; within a group, bands of BAND row tiles, in a band n tile by
// n tile (neighbouring CTAs share a tile of w, and a band's rows stay in L2 while
// all of w passes). A group's rows are spread evenly over its row tiles.
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
    int tl = w - ts[lo] * n_tiles;
    const int band = tl / (BAND * n_tiles);
    tl -= band * BAND * n_tiles;
    const int in_band = min(BAND, mt - band * BAND);
    const int n_tile = tl / in_band;
    const int m_tile = band * BAND + tl - n_tile * in_band;
    const int rows = offs[lo + 1] - offs[lo];
    const int per = ((rows + mt - 1) / mt + ROW_STEP - 1) / ROW_STEP * ROW_STEP;
    r.row0 = offs[lo] + m_tile * per;
    r.rows = min(per, offs[lo + 1] - r.row0);
    r.n0 = n_tile * BM;
    return r;
}

__device__ __forceinline__ float gelu(float x) { return 0.5f * x * erfcf(x * -0.70710678118654752440f); }
// 0.5 x (1 + tanh(u)) = x / (1 + e^(-2u)), u = sqrt(2/pi) (x + 0.044715 x^3)
__device__ __forceinline__ float gelu_tanh(float x)
{
    const float u2 = x * fmaf(0.071354816272600125f, x * x, 1.5957691216057308f);
    return __fdividef(x, 1.0f + __expf(-u2));
}
__device__ __forceinline__ float silu_of(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

template <int N>
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
        for (int i = 0; i < N; ++i) v[i] = gelu(v[i]);
        break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = gelu_tanh(v[i]);
        break;
    default: break;
    }
}

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

template <typename OUT, int BN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
linear_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_a_small,
              const __grid_constant__ CUtensorMap tm_w, const LinearArgs args)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t tiles_addr = (raw_addr + 1023u) & ~1023u;
    using C = Cfg<BN>;
    constexpr int HALF = BN / 2;       // rows of an epilogue thread
    constexpr int STAGES = C::STAGES;
    SmemTail<STAGES>* st =
        reinterpret_cast<SmemTail<STAGES>*>(smem_raw + (tiles_addr - raw_addr) + (size_t)STAGES * C::STAGE_BYTES);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = args.G;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&st->full[s]), 1);
            mbar_init(smem_u32(&st->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&st->tfull[a]), 1);
            mbar_init(smem_u32(&st->tempty[a]), EPI_WARPS);
        }
        mbar_init(smem_u32(&st->drain), 1);
        st->abort = 0;
        fence_barrier_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_a_small);
        tma_prefetch_desc(&tm_w);
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(&st->tmem_base), C::TMEM_COLS);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {
        // the row tiles before each group (a scan, 32 groups at a time); offsets that
        // decrease or leave [0, R] are reported and give no tiles at all, so no row
        // outside the operands is touched
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
                n = good ? (end - first + BN - 1) / BN : 0;
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
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = st->tmem_base;
    const int n_tiles = (args.N + BM - 1) / BM;
    const int k_blocks = (args.K + BK - 1) / BK;
    const int tiles = st->tile_start[G] * n_tiles;
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
                for (int w = blockIdx.x; ok && w < tiles; w += gridDim.x) {
                    const Tile it = decode_tile(w, n_tiles, st->tile_start, st->offsets, G);
                    // boxes of 128 rows, then of 32 up to the tile's last row
                    const int large = it.rows / kLinearRowBox;
                    const int small = (it.rows - large * kLinearRowBox + kLinearRowBoxSmall - 1) / kLinearRowBoxSmall;
                    const uint32_t bytes = W_BYTES + (uint32_t)(large * kLinearRowBox + small * kLinearRowBoxSmall) * BK * 2;
                    for (int kb = 0; kb < k_blocks; ++kb) {
                        if (!mbar_wait(smem_u32(&st->empty[stage]), phase ^ 1u, abort, args.err)) {
                            ok = false;
                            break;
                        }
                        const uint32_t full = smem_u32(&st->full[stage]);
                        const uint32_t w_dst = tiles_addr + stage * C::STAGE_BYTES;
                        uint32_t a_dst = w_dst + W_BYTES;
                        mbar_arrive_expect_tx(full, bytes);
                        if (args.w_nk) {
                            tma_load_3d(w_dst, &tm_w, kb * BK, it.n0, it.g, full);
                        } else {
                            tma_load_3d(w_dst, &tm_w, it.n0, kb * BK, it.g, full);
                            tma_load_3d(w_dst + W_BYTES / 2, &tm_w, it.n0 + 64, kb * BK, it.g, full);
                        }
                        int row = it.row0;
                        for (int i = 0; i < large; ++i, row += kLinearRowBox, a_dst += kLinearRowBox * BK * 2)
                            tma_load_2d(a_dst, &tm_a, kb * BK, row, full);
                        for (int i = 0; i < small; ++i, row += kLinearRowBoxSmall, a_dst += kLinearRowBoxSmall * BK * 2)
                            tma_load_2d(a_dst, &tm_a_small, kb * BK, row, full);
                        ++issued;
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    }
                }
                if (!ok) {
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
            // the whole warp walks the tiles and waits (uniform control flow, so the
            // descriptors stay in uniform registers); one elected lane issues
            const uint32_t leader = elect_one_sync();
            // w with contiguous n: 64 n x 8 k atoms, the second 64 n 8 KB on, a K step of
            // 16 rows of 128 bytes; with contiguous k (as a): 32 bytes along the row
            const uint64_t w_desc = args.w_nk ? smem_desc_sw128(tiles_addr, 16, 1024)
                                              : smem_desc_sw128(tiles_addr, W_BYTES / 2, 1024);
            const uint64_t w_step = args.w_nk ? 2 : 16 * 128 / 16;
            const uint64_t a_desc = smem_desc_sw128(tiles_addr + W_BYTES, 16, 1024);
            const uint32_t fmt = args.fp16 ? 0u : 1u;
            const uint32_t idesc0 = (1u << 4) | (fmt << 7) | (fmt << 10) | ((args.w_nk ? 0u : 1u) << 15) | ((BM >> 4) << 24);
            int stage = 0;
            uint32_t phase = 0;
            int buf = 0;
            uint32_t buf_phase = 0;
            bool ok = true;
            bool any = false;
            for (int w = blockIdx.x; ok && w < tiles; w += gridDim.x) {
                const Tile it = decode_tile(w, n_tiles, st->tile_start, st->offsets, G);
                const uint32_t idesc = idesc0 | ((uint32_t)((it.rows + ROW_STEP - 1) / ROW_STEP * ROW_STEP >> 3) << 17);
                for (int kb = 0; kb < k_blocks; ++kb) {
                    const bool opens = kb % STRETCH == 0;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(smem_u32(&st->full[stage]), phase, abort, args.err) &&
                                        (!opens || mbar_wait(smem_u32(&st->tempty[buf]), buf_phase ^ 1u, abort, args.err)));
                    if (!ok) break;
                    tc_fence_after();
                    const bool closes = kb % STRETCH == STRETCH - 1 || kb == k_blocks - 1;
                    if (leader) {
                        const uint32_t d = tmem_base + buf * BN;
                        const uint64_t at = (uint64_t)(stage * (C::STAGE_BYTES >> 4));
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            tc_mma_f16(d, w_desc + at + w_step * kk, a_desc + at + 2 * kk, idesc, !opens || kk != 0 ? 1u : 0u);
                        tc_commit(smem_u32(&st->empty[stage]));
                        if (closes) tc_commit(smem_u32(&st->tfull[buf]));
                    }
                    __syncwarp();
                    any = true;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (closes && ++buf == 2) { buf = 0; buf_phase ^= 1u; }
                }
            }
            if (!ok && any && leader) {
                // drain: every MMA issued so far must finish before TMEM is freed
                tc_commit(smem_u32(&st->drain));
                mbar_wait_drain(smem_u32(&st->drain), 0);
            }
            __syncwarp();
        }
    } else {
        setmaxnreg_inc<EPI_REGS>();
        // ============================== epilogue ==============================
        const int c0 = (warp >> 2) * HALF;             // this thread's rows of the tile
        const uint32_t t_row = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + c0;
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < tiles; w += gridDim.x) {
            const Tile it = decode_tile(w, n_tiles, st->tile_start, st->offsets, G);
            const int rows = it.rows - c0;             // of them there are so many
            float acc[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) acc[i] = 0.0f;
            for (int kb = 0; kb < k_blocks; kb += STRETCH) {
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
                if (lane == 0) mbar_arrive(smem_u32(&st->tempty[buf]));
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            }
            if (!ok) break;
            const int n = it.n0 + (warp & 3) * 32 + lane;
            if (n < args.N) {
                float bias = 0.0f;
                if (args.bias) {
                    const int64_t at = (int64_t)it.g * args.N + n;
                    bias = args.bias_f32 ? __ldg(static_cast<const float*>(args.bias) + at)
                           : args.fp16   ? __half2float(static_cast<const __half*>(args.bias)[at])
                                         : __bfloat162float(static_cast<const __nv_bfloat16*>(args.bias)[at]);
                }
                OUT* out = static_cast<OUT*>(args.out) + (int64_t)(it.row0 + c0) * args.out_stride + n;
                const OUT* res = static_cast<const OUT*>(args.residual);
                if (res) res += (int64_t)(it.row0 + c0) * args.residual_stride + n;
#pragma unroll
                for (int c = 0; c < HALF; c += 32) {
                    if (c >= rows) break;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = acc[c + i] + bias;
                    activate(v, args.act);
                    if (res) {
                        OUT r[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < rows) r[i] = res[(c + i) * args.residual_stride];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += as_float(r[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c + i < rows) put(out + (c + i) * args.out_stride, v[i]);
                }
            }
        }
    }

    // ---- teardown: every role is done (or has drained after an abort)
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

constexpr int kMaxDevices = 64;

template <typename OUT, int BN>
cudaError_t launch(const CUtensorMap& tm_a, const CUtensorMap& tm_a_small, const CUtensorMap& tm_w, const LinearArgs& a,
                   int num_sms, cudaStream_t s)
{
    auto kern = linear_kernel<OUT, BN>;
    constexpr size_t smem = smem_bytes<BN>();
    // asked of the runtime once per kernel and device
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const uint64_t bit = (uint64_t)1 << dev;
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    return launch_pdl(kern, dim3((unsigned)num_sms), dim3(NUM_THREADS), smem, s, tm_a, tm_a_small, tm_w, a);
}

template <typename OUT>
cudaError_t launch_out(const CUtensorMap& tm_a, const CUtensorMap& tm_a_small, const CUtensorMap& tm_w,
                       const LinearArgs& a, int num_sms, cudaStream_t s)
{
    if ((int64_t)a.R <= (int64_t)128 * a.G) return launch<OUT, 128>(tm_a, tm_a_small, tm_w, a, num_sms, s);
    return launch<OUT, 256>(tm_a, tm_a_small, tm_w, a, num_sms, s);
}

}  // namespace

cudaError_t launch_linear(moe_dtype out_dtype, const CUtensorMap& tm_a, const CUtensorMap& tm_a_small,
                          const CUtensorMap& tm_w, const LinearArgs& a, int num_sms, cudaStream_t s)
{
    if (a.R == 0) return cudaSuccess;
    if (a.R < 0 || a.G < 1 || a.G > MAX_GROUPS || (!a.offsets && a.G != 1)) return cudaErrorInvalidValue;
    switch (out_dtype) {
    case MOE_BF16: return launch_out<__nv_bfloat16>(tm_a, tm_a_small, tm_w, a, num_sms, s);
    case MOE_FP16: return launch_out<__half>(tm_a, tm_a_small, tm_w, a, num_sms, s);
    case MOE_FP32: return launch_out<float>(tm_a, tm_a_small, tm_w, a, num_sms, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
