/*
 * moe.h -- C ABI of the GB300 (sm_103a) MoE FFN layer forward.
 *
 * The layer: top-k routing, dispatch of the routed (token, expert) pairs into
 * per-expert groups, a SwiGLU expert FFN per group (GEMM0 + SwiGLU split
 * along the token dimension M, GEMM1 split along the hidden dimension N),
 * and the gate-weighted combine back to token order. The parts are those
 * named in the DisagMoE summary (gist.science, "Resumo Tecnico: DisagMoE",
 * section 2.2, "Alinhamento de Estagios": top-k experts, dispatch, combine)
 * and on the COMET page (nav.superapi.store/en/comet, "COMET's Technical
 * Principles", "Tensor Decomposition": Layer 0 split along M, Layer 1 along
 * N). The pages give no formulas; the readings used here are:
 *   - logits l[t,e] = sum_h x[t,h] Wg[h,e] in fp32 in one canonical order
 *     (8-element chunks, chunk c on lane c mod 32, fma in increasing h, then
 *     an xor butterfly over the 32 lane sums with strides 16, 8, 4, 2, 1),
 *     plus bias[e] when a bias is given;
 *   - top-k on the logits, descending, ties to the lower expert id; the rank
 *     of an expert is its selection position;
 *   - gate weights = softmax over the k selected logits;
 *   - expert e: y = (silu(x W1[e]) * (x W3[e])) W2[e], silu(a) = a/(1+e^-a);
 *   - out[t] = sum over ranks j = 0..k-1 (in that order) of w[t,j] y_j,
 *     plus the always-on shared expert (weight 1) when F_shared > 0.
 *
 * Conventions (every entry point):
 *   - Tensors are row-major and contiguous: x[T,H], Wg[H,E], W1/W3[E,H,F],
 *     W2[E,F,H]; shared expert W1s/W3s[H,Fs], W2s[Fs,H]. bf16 tensors are
 *     passed as moe_bf16 (raw bf16 bits).
 *   - Every pointer is a device pointer owned by the caller; the library
 *     allocates no memory and keeps no per-call state. Scratch memory is the
 *     caller's workspace `ws` of at least moe_workspace_size(dims) bytes,
 *     256-byte aligned. Two calls that share a workspace must not overlap.
 *   - Calls are asynchronous on `stream`. Argument checks run on the host
 *     before any launch and return MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED
 *     / MOE_ERR_WORKSPACE without launching. A launch failure returns
 *     MOE_ERR_CUDA. Errors found on the device (an expert id outside
 *     [0, E), a bounded wait that ran out) are OR-ed into the error word at
 *     the start of `ws` and read by moe_check(); with the environment
 *     variable MOE_DEBUG=1 every entry point synchronises and checks.
 *   - Supported shapes (else MOE_ERR_UNSUPPORTED): 1 <= k <= min(E, 8),
 *     E <= 256, H and F (and F_shared) multiples of 64, T*k < 2^31.
 *     T == 0 is a valid no-op. Pointers must be 16-byte aligned.
 *   - Results are bit-identical from run to run (no float atomics).
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t moe_bf16;                 /* raw bf16 bits */
typedef uint8_t moe_e4m3;                  /* raw 8-bit floating-point bits: 1 sign, 4 exponent, 3 mantissa */
typedef struct CUstream_st* moe_stream_t;  /* the same type as cudaStream_t */
typedef struct CUevent_st* moe_event_t;    /* the same type as cudaEvent_t */

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* null pointer, negative size, bad id (device) */
    MOE_ERR_UNSUPPORTED = 2,   /* shape outside the supported set */
    MOE_ERR_WORKSPACE = 3,     /* workspace missing, too small or misaligned */
    MOE_ERR_CUDA = 4,          /* a CUDA runtime / driver call failed */
    MOE_ERR_TIMEOUT = 5,       /* a bounded device wait ran out (device) */
    MOE_ERR_DEVICE_BOUNDS = 6  /* a device index check failed (device) */
} moe_status;

/* Element types of the entry points that take more than one. */
typedef enum { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 } moe_dtype;

typedef struct {
    int64_t T;         /* tokens */
    int32_t H;         /* hidden size */
    int32_t F;         /* expert FFN width */
    int32_t E;         /* routed experts */
    int32_t k;         /* experts per token */
    int32_t F_shared;  /* shared expert FFN width; 0 = no shared expert */
} moe_dims;

/* Optional per-stage timing: each non-null event is recorded on the stream
 * at that point of moe_layer_forward. */
typedef struct {
    moe_event_t before_route;
    moe_event_t before_permute;
    moe_event_t before_gemm0;      /* routed GEMM0 + SwiGLU */
    moe_event_t before_gemm1;      /* routed GEMM1 + weighted scatter */
    moe_event_t before_shared;     /* shared-expert GEMM0 + GEMM1 (if any) */
    moe_event_t before_combine;
    moe_event_t after_combine;
} moe_stage_events;

/* Gating variants (readings of this library; the pages give no gate formula).
 * A null moe_gating* means {renormalize = 1, shared_gate = NULL}. */
typedef struct {
    int32_t renormalize;          /* 1: weights = softmax over the k selected logits;
                                     0: softmax over all E logits at the selected ids
                                        (the k weights then sum to less than 1) */
    const moe_bf16* shared_gate;  /* [H] or NULL: scale the shared expert's output by
                                     sigmoid(x[t] . shared_gate) instead of 1 */
} moe_gating;

/* Optional routing outputs of moe_layer_forward; each null field is kept in
 * the workspace instead. Sizes: [T*k], [T*k], [E], [E+1], [T*k], [T*k]. */
typedef struct {
    int32_t* topk_idx;
    float* topk_w;
    int32_t* counts;
    int32_t* offsets;
    int32_t* src_row;
    int32_t* inv_pos;
} moe_routing_out;

/* Library-wide options (moe_set_option / moe_get_option). */
enum {
    /* How GEMM0 obtains the routed token rows (its A operand):
     *   MOE_GEMM0_A_PERMUTED   (default) the dispatch step copies them into
     *                          dispatch order (x_perm, in the workspace) and
     *                          GEMM0 loads dense 128-row TMA tiles;
     *   MOE_GEMM0_A_TMA_GATHER the GEMM0 producer warp gathers them straight
     *                          from x with TMA gather4, 4 rows per instruction;
     *   MOE_GEMM0_A_CP_GATHER  a GEMM0 producer warp gathers them straight
     *                          from x with 16-byte cp.async copies.
     * All give bit-identical results. */
    MOE_OPT_GEMM0_A = 0,
    MOE_GEMM0_A_PERMUTED = 0,
    MOE_GEMM0_A_TMA_GATHER = 1,
    MOE_GEMM0_A_CP_GATHER = 2,
    /* Where moe_layer_forward sums the k weighted expert rows of a token:
     *   MOE_COMBINE_AUTO     (default) fused when the last GEMM1 to run (the
     *                        shared expert's if any, else the routed one) has
     *                        K >= 4096, else separate;
     *   MOE_COMBINE_FUSED    in GEMM1's epilogue: each row takes an integer
     *                        ticket per (token, 256-column tile) and the last
     *                        one sums the token's slots in rank order;
     *   MOE_COMBINE_SEPARATE a streaming combine kernel after the GEMMs.
     * Both sum the same fp32 values in the same order: bit-identical. */
    MOE_OPT_COMBINE = 1,
    MOE_COMBINE_AUTO = 0,
    MOE_COMBINE_FUSED = 1,
    MOE_COMBINE_SEPARATE = 2,
    /* Whether moe_layer_forward runs the routed experts' two GEMMs as one
     * persistent launch (GEMM1 tiles start as soon as the GEMM0 tiles of their
     * expert and 128-row block have written h; no launch boundary, no GEMM0
     * tail) or as two launches. Only with MOE_GEMM0_A_PERMUTED.
     *   MOE_GEMM_FUSION_AUTO (default) the table in the library's layer call
     *                        (by shape; see moe_layer_forward);
     *   MOE_GEMM_FUSION_ON / MOE_GEMM_FUSION_OFF force it.
     * Same arithmetic either way: bit-identical. */
    MOE_OPT_GEMM_FUSION = 2,
    MOE_GEMM_FUSION_AUTO = 0,
    MOE_GEMM_FUSION_ON = 1,
    MOE_GEMM_FUSION_OFF = 2,
    /* How many CTAs share one tensor-core MMA in the expert GEMMs that read a
     * dense A operand (GEMM0 over x_perm, every GEMM1, the shared expert):
     *   MOE_CTA_GROUP_AUTO (default) the table in the library's layer call
     *                      (by rows per expert and GEMM; see moe_layer_plan);
     *   MOE_CTA_GROUP_ONE  one CTA per 128 x 256 MMA tile;
     *   MOE_CTA_GROUP_PAIR a 2-CTA cluster per 256 x 256 MMA tile
     *                      (tcgen05 cta_group::2): each CTA stages 128 rows
     *                      of A and half of B's columns.
     * The gathered GEMM0 forms and the one-launch GEMM pair always run one CTA
     * per MMA. */
    MOE_OPT_CTA_GROUP = 3,
    MOE_CTA_GROUP_AUTO = 0,
    MOE_CTA_GROUP_ONE = 1,
    MOE_CTA_GROUP_PAIR = 2,
    /* Who copies the routed token rows into dispatch order (x_perm) when
     * GEMM0 reads them from there (MOE_GEMM0_A_PERMUTED, two GEMM launches):
     *   MOE_X_PERM_COPY_AUTO   (default) the table (see moe_layer_plan): the
     *                          kernel, which measured as fast on GB300;
     *   MOE_X_PERM_COPY_INLINE a spare warp of every GEMM0 CTA, while the
     *                          GEMM runs: each 128-row tile is computed as
     *                          soon as its rows are copied (counted per
     *                          tile), so the copy overlaps the tensor work;
     *   MOE_X_PERM_COPY_KERNEL a copy kernel before GEMM0.
     * The same bytes either way: bit-identical. */
    MOE_OPT_X_PERM_COPY = 4,
    MOE_X_PERM_COPY_AUTO = 0,
    MOE_X_PERM_COPY_INLINE = 1,
    MOE_X_PERM_COPY_KERNEL = 2,
    /* Which router moe_layer_forward runs:
     *   MOE_ROUTER_OPT_AUTO   (default) the table (see moe_layer_plan): the
     *                         tensor-core router for 16 <= E <= 64 (E a
     *                         multiple of 8) from T = 8192, where it measured
     *                         faster, else an FMA router;
     *   MOE_ROUTER_OPT_FMA    the FMA routers (the canonical order itself);
     *   MOE_ROUTER_OPT_TENSOR the tensor-core router wherever it applies
     *                         (8 <= E <= 64, E a multiple of 8, T >= 512).
     * The expert ids and their order are the same bit for bit either way
     * (the tensor-core router proves each token's selection against the
     * canonical order, or recomputes the token in it); the gate weights agree
     * to fp32 rounding (a softmax of logits whose summation order differs). */
    MOE_OPT_ROUTER = 5,
    MOE_ROUTER_OPT_AUTO = 0,
    MOE_ROUTER_OPT_FMA = 1,
    MOE_ROUTER_OPT_TENSOR = 2
};

/* Sets a library-wide option for later calls (all devices and threads).
 * Returns MOE_ERR_INVALID_ARG for an unknown option or value. Do not change
 * options while another thread is inside a call. */
moe_status moe_set_option(int option, int value);

/* Current value of an option, or -1 for an unknown option. */
int moe_get_option(int option);

/* Router kernels (moe_plan.router). All select the same experts in the same
 * order bit for bit; the FMA routers (0..3) also give the same logits. */
enum {
    MOE_ROUTER_STREAM = 0,   /* E <= 8: TMA-fed per-warp pipelines, top-k fused */
    MOE_ROUTER_SLICED = 1,   /* E > 8, a multiple of 8, inside moe_layer_forward: expert
                              * slices of 8 per CTA, logits to the workspace, top-k pass */
    MOE_ROUTER_CLUSTER = 2,  /* 8 < E <= 64: canonical lanes split over a CTA cluster */
    MOE_ROUTER_BLOCK = 3,    /* anything else: one CTA per SM, gate staged in slices */
    MOE_ROUTER_TENSOR = 4    /* inside moe_layer_forward, 8 <= E <= 64, E % 8 == 0: the
                              * gate GEMM on tcgen05; each token's top-k proven equal to
                              * the canonical order's by an error bound (ties and near
                              * ties recomputed in the canonical order) */
};

/* The configuration moe_layer_forward runs for a shape under the current
 * options: the library's per-shape table, fixed before any launch. */
typedef struct {
    int32_t router;        /* MOE_ROUTER_* */
    int32_t gemm0_a;       /* MOE_GEMM0_A_* in effect */
    int32_t combine;       /* MOE_COMBINE_FUSED or MOE_COMBINE_SEPARATE */
    int32_t gemm_fusion;   /* MOE_GEMM_FUSION_ON or MOE_GEMM_FUSION_OFF */
    int32_t tile_m;        /* grouped GEMM tile rows (routed rows per tile; 256 for a CTA pair) */
    int32_t tile_n;        /* grouped GEMM MMA N (GEMM0: half W1, half W3) */
    int32_t tile_k;        /* K per pipeline stage */
    int32_t stages;        /* shared-memory pipeline stages */
    int32_t cta_group;     /* CTAs per MMA (tcgen05 cta_group) of the routed GEMM0; tile_m
                            * and stages describe it */
    int32_t cta_group_gemm1; /* the same for the routed GEMM1 (a second launch; 1 when both
                              * GEMMs share one launch) */
    int32_t x_perm_copy;   /* MOE_X_PERM_COPY_INLINE or _KERNEL; 0 when GEMM0 does not read x_perm */
} moe_plan;

/* Fills *plan for `dims` (host only: no device work, no launch). Returns
 * MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED for shapes moe_layer_forward
 * rejects. */
moe_status moe_layer_plan(const moe_dims* dims, moe_plan* plan);

/* Self-test of the failure path every pipeline wait takes: one device thread
 * waits, bounded by limit_ms (1..4000) of %globaltimer time, on a device flag
 * that nothing sets, gives up, and reports it through a device error word.
 * Returns MOE_ERR_TIMEOUT when that happened (the expected outcome), MOE_OK if
 * the wait somehow completed, MOE_ERR_CUDA on a launch or copy error. The
 * device stays usable. Synchronises `stream`. */
moe_status moe_selftest_wait_timeout(int32_t limit_ms, moe_stream_t stream);

/* Test hook: one device thread that sleeps for `ms` (1..6000) of %globaltimer
 * time and lets the next kernel of the stream become resident meanwhile. Does
 * not synchronise. */
moe_status moe_selftest_hold(int32_t ms, moe_stream_t stream);

/* Test hook of the tensor-core router (MOE_ROUTER_TENSOR): routes x with it
 * as moe_layer_forward would, writing topk_idx[T,k] / topk_w[T,k] and
 * optionally
 *   fast_logits[T,E]  the tensor-core logits (before the bias),
 *   fast_bound[T]     the bound used for the tensor-core part of the error,
 *                     c_fast ||x_t|| max_e ||w_e||, so that a caller can check
 *                     |fast_logits - exact| <= fast_bound,
 *   n_exact           how many tokens took the canonical recomputation
 *                     (reading it synchronises `stream`).
 * force_exact != 0 sends every token through the canonical recomputation.
 * ws is a moe_layer_forward workspace for dims. MOE_ERR_UNSUPPORTED where the
 * tensor-core router does not apply. Not needed for normal use. */
moe_status moe_selftest_route_tc(const moe_dims* dims, const moe_bf16* x, const moe_bf16* Wg,
                                 const float* bias, int32_t renormalize, int32_t force_exact,
                                 int32_t* topk_idx, float* topk_w, float* fast_logits,
                                 float* fast_bound, int64_t* n_exact, void* ws, size_t ws_bytes,
                                 moe_stream_t stream);

/* Library version (major*10000 + minor*100 + patch). */
int moe_version(void);

/* Number of CUDA kernels this library has launched in this process (all
 * threads, devices and streams) since it was loaded: each kernel launch of
 * every call counts once; memsets and copies do not. A caller takes the
 * difference around a region to count what that region launched. */
uint64_t moe_launch_count(void);

/* Text for a status code. Never null. */
const char* moe_status_string(int status);

/* Workspace bytes that every entry point below accepts for `dims`.
 * Returns 0 for invalid dims. */
size_t moe_workspace_size(const moe_dims* dims);

/* Synchronises `stream`, reads and clears the device error word at the start
 * of `ws`, and returns the status it holds (MOE_OK if none). */
moe_status moe_check(void* ws, moe_stream_t stream);

/*
 * Router (top-k gating).
 * In:  x[T,H], Wg[H,E] (bf16); bias[E] (f32, may be null).
 * Out: topk_idx[T,k] (int32, expert ids in rank order), topk_w[T,k] (f32,
 *      the softmax of the selected logits, in rank order).
 * The logits are computed in the canonical fp32 order given above, so the ids
 * are bit-exact against any implementation of that order.
 */
moe_status moe_route(const moe_dims* dims, const moe_bf16* x, const moe_bf16* Wg, const float* bias,
                     int32_t* topk_idx, float* topk_w, moe_stream_t stream);

/* moe_route with a gating variant (gating->renormalize; shared_gate unused). */
moe_status moe_route_ex(const moe_dims* dims, const moe_bf16* x, const moe_bf16* Wg, const float* bias,
                        const moe_gating* gating, int32_t* topk_idx, float* topk_w, moe_stream_t stream);

/*
 * Dispatch: stable counting sort of the R = T*k assignments f = t*k + j by
 * expert id topk_idx[f] (the "dispatch" of the DisagMoE summary, 2.2).
 * In:  topk_idx[R] (int32).
 * Out: counts[E]; offsets[E+1] (exclusive scan, offsets[E] = R);
 *      src_row[R] (src_row[p] = f, experts in increasing order, f increasing
 *      within an expert); inv_pos[R] (inv_pos[f] = p).
 *      x_perm[R,H] (may be null): x_perm[p] = x[src_row[p] / k]; x must be
 *      given when x_perm is. (Rows are copied as they are: bf16, or fp16
 *      behind the same pointers.)
 * An id outside [0, E) sets MOE_ERR_INVALID_ARG in the device error word and
 * that assignment is skipped (no out-of-bounds write).
 * Also writes the GEMM tile table into `ws` for a later moe_expert_ffn /
 * moe_layer_forward on the same workspace.
 */
moe_status moe_permute(const moe_dims* dims, const int32_t* topk_idx, int32_t* counts,
                       int32_t* offsets, int32_t* src_row, int32_t* inv_pos, const moe_bf16* x,
                       moe_bf16* x_perm, void* ws, size_t ws_bytes, moe_stream_t stream);

/*
 * Dispatch with no workspace: the same results as moe_permute (counts,
 * offsets, src_row, inv_pos and the optional x_perm, bit for bit), for
 * callers that cannot provide scratch memory -- a host framework that gives
 * its plug-ins no allocator or scratch hook, or a service whose device memory
 * budget is fixed at start-up and which must not allocate while serving.
 * The pages have no counterpart to this entry point; it is an interface
 * convenience of this library.
 * Scratch: a fixed 1 MiB array inside the library, one per GPU, held until
 * the process exits. Shapes whose per-chunk histogram (ceil(T*k / 2048) * E
 * ints) exceeds 261632 ints are rejected with MOE_ERR_UNSUPPORTED before any
 * launch (for example E = 64 allows T*k up to 8,372,224).
 * The first call on a device looks up the array's device address with that
 * device current; make it before any stream capture on the device. The
 * address is cached for the life of the device's context: calling
 * cudaDeviceReset after the first call is not supported. All calls
 * on a device share the array, which keeps the last call's contents (nothing
 * in it needs to start at zero); calls that overlap on the GPU race on it and
 * must be serialised by the caller. No memory is allocated by this call.
 * The shape checks are moe_permute's. An expert id outside [0, E) is
 * skipped (offsets[E] then ends below T*k); there is no device error word.
 * With MOE_DEBUG=1 the call synchronises and returns MOE_ERR_CUDA if a
 * launch faulted.
 */
moe_status moe_permute_static(const moe_dims* dims, const int32_t* topk_idx, int32_t* counts,
                              int32_t* offsets, int32_t* src_row, int32_t* inv_pos,
                              const moe_bf16* x, moe_bf16* x_perm, moe_stream_t stream);

/*
 * Expert FFN over the dispatched groups: for every position p of expert e
 * (offsets[e] <= p < offsets[e+1]) with f = src_row[p], t = f / k, j = f % k:
 *   h[p]      = silu(x[t] W1[e]) * (x[t] W3[e])     (GEMM0 + SwiGLU, h in bf16)
 *   slot[j,t] = w * (h[p] W2[e])                    (GEMM1 + weighted scatter)
 * with w = topk_w[f], or 1 when topk_w is null.
 * In:  x[T,H]; src_row[R] (null = identity: f = p); offsets[E+1] (null = one
 *      group holding all R rows; then E must be 1); W1/W3[E,H,F], W2[E,F,H].
 * Out: slot[k,T,H] (f32). Every (j, t) slot is written exactly once.
 * Call with dims {T, H, F=Fs, E=1, k=1} and null src_row/offsets/topk_w to
 * run a dense (shared) expert into slot[0].
 */
moe_status moe_expert_ffn(const moe_dims* dims, const moe_bf16* x, const int32_t* src_row,
                          const int32_t* offsets, const moe_bf16* W1, const moe_bf16* W3,
                          const moe_bf16* W2, const float* topk_w, float* slot, void* ws,
                          size_t ws_bytes, moe_stream_t stream);

/*
 * Combine (the "combine" of the DisagMoE summary, 2.2): out[t,:] =
 * bf16( ((slot[0,t,:] + slot[1,t,:]) + ...) + slot[n_slots-1,t,:] ), an fp32
 * left fold in slot order, no atomics.
 * In:  slot[n_slots,T,H] (f32), 1 <= n_slots <= 9.  Out: out[T,H] (bf16).
 */
moe_status moe_combine(const moe_dims* dims, const float* slot, int32_t n_slots, moe_bf16* out,
                       moe_stream_t stream);

/*
 * The whole layer: route -> permute -> expert FFN (routed; then the shared
 * expert when dims->F_shared > 0) -> combine.
 * In:  x, Wg, bias (nullable), W1, W3, W2; W1s/W3s/W2s (needed iff F_shared > 0).
 * Out: out[T,H] (bf16); routing (nullable) receives the routing tensors.
 * events (nullable) are recorded at the stage boundaries.
 */
moe_status moe_layer_forward(const moe_dims* dims, const moe_bf16* x, const moe_bf16* Wg,
                             const float* bias, const moe_bf16* W1, const moe_bf16* W3,
                             const moe_bf16* W2, const moe_bf16* W1s, const moe_bf16* W3s,
                             const moe_bf16* W2s, moe_bf16* out, const moe_routing_out* routing,
                             void* ws, size_t ws_bytes, const moe_stage_events* events,
                             moe_stream_t stream);

/* moe_layer_forward with a gating variant (nullable; see moe_gating). A
 * shared_gate needs F_shared > 0; its [H] vector must be 16-byte aligned. */
moe_status moe_layer_forward_ex(const moe_dims* dims, const moe_bf16* x, const moe_bf16* Wg,
                                const float* bias, const moe_gating* gating, const moe_bf16* W1,
                                const moe_bf16* W3, const moe_bf16* W2, const moe_bf16* W1s,
                                const moe_bf16* W3s, const moe_bf16* W2s, moe_bf16* out,
                                const moe_routing_out* routing, void* ws, size_t ws_bytes,
                                const moe_stage_events* events, moe_stream_t stream);

/*
 * The whole layer from and to host memory: x_host[T,H] in, out_host[T,H] out
 * (bf16), every weight already on the device. The tokens are split into
 * n_chunks consecutive chunks (0: the library's choice, else 1..64) and the
 * chunks are pipelined: while the layer runs on chunk c (on `stream`), the
 * host-to-device copy of chunk c+1 and the device-to-host copy of chunk c-1
 * run on two copy streams the library keeps per device. Tokens are
 * independent (routing and the expert GEMMs of a row do not depend on the
 * other rows in its chunk) and every chunk runs the router family the whole
 * batch would, so every output row is bit for bit the one moe_layer_forward
 * gives for the whole batch. One exception: when the whole batch takes the
 * tensor-core router and a caller-chosen n_chunks leaves a chunk below the
 * 512 tokens that router needs, that chunk takes the FMA routers: the same
 * ids and dispatch, gate weights within fp32 rounding (the library's own
 * chunk choice never does this).
 *
 * x_host and out_host should be page-locked (cudaHostAlloc /
 * cudaHostRegister); pageable memory works but its copies do not overlap.
 * x_dev and out_dev are caller-owned device staging buffers of T*H bf16
 * each, 16-byte aligned; on return x_dev holds x and out_dev the output.
 * ws is moe_workspace_size(dims) bytes (the whole batch's), as for
 * moe_layer_forward. The call is stream-ordered on `stream`: it starts after
 * the work already queued there, and work queued there afterwards starts
 * once out_host holds the result (synchronize the stream before reading it).
 * Errors: the argument checks of moe_layer_forward (MOE_ERR_INVALID_ARG for
 * a null or misaligned pointer or n_chunks outside 0..64); MOE_ERR_CUDA if a
 * copy, an event or a launch fails, after which out_host is unspecified (work
 * queued on `stream` afterwards still waits for every copy already queued).
 * Concurrent calls from several host threads on one device share the copy
 * streams and are serialized by them (correct, not overlapped).
 */
moe_status moe_layer_forward_host(const moe_dims* dims, const moe_bf16* x_host, const moe_bf16* Wg,
                                  const float* bias, const moe_bf16* W1, const moe_bf16* W3,
                                  const moe_bf16* W2, const moe_bf16* W1s, const moe_bf16* W3s,
                                  const moe_bf16* W2s, moe_bf16* out_host, moe_bf16* x_dev,
                                  moe_bf16* out_dev, int32_t n_chunks, void* ws, size_t ws_bytes,
                                  moe_stream_t stream);

/* The chunk count moe_layer_forward_host uses for n_chunks = 0 (host only). */
int32_t moe_host_chunks(const moe_dims* dims);

/*
 * ------------------------------------------------------------------ 8 bits --
 * The layer with its expert products in 8-bit floating point. A value v is
 * held as e4m3 q with its block's fp32 scale, v = q * scale:
 *   activations [R, n]: a scale for each row's block of 128 columns,
 *                       scale[R, ceil(n/128)];
 *   weights [G, N, K]:  a scale for each 128 x 128 block, scale[G, ceil(N/128),
 *                       ceil(K/128)]. K is contiguous (the transpose of the
 *                       bf16 weights above).
 * Quantizing a block: scale = max(largest |v|, 2^-100) / 448, and q the nearest
 * e4m3 (ties to even) to v / scale for weights, to v * (1 / scale) for
 * activations, each operation rounded to fp32; a NaN or infinity in a block makes
 * all of it NaN or is carried as NaN. Sizes are multiples of 16, the last block may be shorter.
 * The products accumulate in fp32 and apply the scales in fp32.
 *
 * Conventions are those of the other entry points. The workspace `ws` of the
 * products (moe_fp8_workspace_size(NULL) bytes, for any sizes) and of
 * moe_fp8_layer_forward (moe_fp8_workspace_size(dims)) must hold zeros in its
 * first MOE_FP8_WORKSPACE_ZEROS bytes (the error word and the tickets of cut
 * tiles) before its first use, and again after moe_check has returned
 * MOE_ERR_TIMEOUT for it; the calls leave them as the next call needs them, of
 * these or any other sizes that the workspace is large enough for. The rest may
 * hold anything. Two calls that share a workspace must not overlap.
 */
#define MOE_FP8_WORKSPACE_ZEROS 2304

/* Bytes of the 8-bit entry points' workspace: of the products for dims NULL,
 * else of moe_fp8_layer_forward (0 for invalid dims). */
size_t moe_fp8_workspace_size(const moe_dims* dims);

/*
 * The residual's addition, the root-mean-square norm and its 8-bit output:
 *   r = x + residual (x where residual is null), in fp32
 *   y = r / sqrt(mean(r^2) + eps) * weight       (weight null = 1), in fp32
 * In:  x[T,H] and residual[T,H] (nullable) of type dtype, rows x_stride and
 *      residual_stride elements apart; weight[H] of type dtype (nullable).
 * Out: sum[T,H] = r rounded to dtype, rows sum_stride apart (nullable; may be
 *      the memory of x or of residual with the same stride); y[T,H] rounded to dtype
 *      (nullable, contiguous); q[T,H] and scale[T,ceil(H/128)]: y quantized
 *      (from fp32, not from its rounding).
 * H a multiple of 16 up to 32768; pointers but scale 16-byte aligned and row
 * strides multiples of 16 bytes, at least H elements. The squares are summed in
 * fp32: a row whose sum passes the largest fp32 (values of 2^64) has y = 0.
 */
moe_status moe_add_rmsnorm_fp8(int64_t T, int32_t H, moe_dtype dtype, const void* x, int64_t x_stride,
                               const void* residual, int64_t residual_stride, const void* weight, float eps, void* sum,
                               int64_t sum_stride, void* y, moe_e4m3* q, float* scale, moe_stream_t stream);

/*
 * A weight's layout for the products, made once: w[G,K,N] (bf16, as the other
 * entry points take them) to q[G,N,K] and its block scales.
 */
moe_status moe_fp8_quantize_weight(int32_t G, int32_t K, int32_t N, const moe_bf16* w, moe_e4m3* q, float* scale,
                                   moe_stream_t stream);

/*
 * Grouped product: out[p,:] = a[p,:] w[g]^T for the rows p of group g,
 * offsets[g] <= p < offsets[g+1] (offsets null = one group of R rows; G is
 * then 1). Rows outside [offsets[0], offsets[G]) are not written. Offsets that
 * decrease or leave [0, R] set MOE_ERR_DEVICE_BOUNDS in the device error word
 * and nothing is computed.
 * In:  a[R,K], a_scale; offsets[G+1] (device); w[G,N,K], w_scale.
 * Out: out[R,N] in bf16 or fp32 (out_dtype).
 */
moe_status moe_fp8_matmul(int64_t R, int32_t K, int32_t N, int32_t G, const moe_e4m3* a, const float* a_scale,
                          const int32_t* offsets, const moe_e4m3* w, const float* w_scale, moe_dtype out_dtype,
                          void* out, void* ws, size_t ws_bytes, moe_stream_t stream);

/*
 * Gated product: h[p,:] = silu(a[p,:] w1[g]^T) * (a[p,:] w3[g]^T) for the rows
 * of each group as in moe_fp8_matmul, both projections, the activation, the
 * product and its quantization in one kernel.
 * In:  a[R,K], a_scale; offsets[G+1]; w1, w3 [G,F,K] and their scales.
 * Out: h[R,F], h_scale[R,ceil(F/128)]: quantized from fp32.
 */
moe_status moe_fp8_gated(int64_t R, int32_t K, int32_t F, int32_t G, const moe_e4m3* a, const float* a_scale,
                         const int32_t* offsets, const moe_e4m3* w1, const float* w1_scale, const moe_e4m3* w3,
                         const float* w3_scale, moe_e4m3* h, float* h_scale, void* ws, size_t ws_bytes,
                         moe_stream_t stream);

/* Test hook (host only): which kernel a product of these sizes (gated != 0: a
 * gated one) runs on a device of num_sms SMs: 0 one CTA per MMA, 1 the same with
 * tiles of 128 columns, 2 a CTA pair; -1 for sizes that the calls refuse. The
 * result does not depend on it but for the order of its sums. */
int32_t moe_selftest_fp8_form(int64_t R, int32_t K, int32_t N, int32_t G, int32_t gated, int32_t num_sms);

/* One expert set's 8-bit weights: w1, w3 [E,F,H], w2 [E,H,F] and their scales
 * (moe_fp8_quantize_weight of W1, W3, W2). */
typedef struct {
    const moe_e4m3* w1;
    const float* w1_scale;
    const moe_e4m3* w3;
    const float* w3_scale;
    const moe_e4m3* w2;
    const float* w2_scale;
} moe_fp8_ffn;

/*
 * The whole layer on 8-bit experts: route (on x in bf16, as moe_layer_forward)
 * -> sort, quantized rows to dispatch order -> gated product -> product,
 * weighted and scattered -> (the shared expert, when F_shared > 0) -> combine.
 * In:  x[T,H] (bf16: the router's input) and the same rows quantized, xq[T,H]
 *      and xq_scale: y, q and scale of moe_add_rmsnorm_fp8; Wg, bias, gating
 *      as in moe_layer_forward_ex; routed (dims->E experts of width F), shared
 *      (one of width F_shared; null without one).
 * Out: out[T,H] (bf16); routing (nullable).
 */
moe_status moe_fp8_layer_forward(const moe_dims* dims, const moe_bf16* x, const moe_e4m3* xq, const float* xq_scale,
                                 const moe_bf16* Wg, const float* bias, const moe_gating* gating,
                                 const moe_fp8_ffn* routed, const moe_fp8_ffn* shared, moe_bf16* out,
                                 const moe_routing_out* routing, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Expert layers of another form: routing from given logits (moe_route_logits),
 * a grouped product with bias, activation and residual (moe_linear), and the
 * weighted sum of the experts' rows (moe_combine_rows). With moe_permute between
 * the first two they are a layer whose router or experts moe_layer_forward does
 * not have. Conventions are those of the other entry points.
 */

/* A router's scores of the logits l[E] of a token: softmax over all E, or 1 / (1 + e^-l). */
typedef enum { MOE_SCORES_SOFTMAX = 0, MOE_SCORES_SIGMOID = 1 } moe_scores;

typedef struct {
    moe_scores scores;
    const float* bias;     /* [E], added to the scores for the selection only; or null */
    int32_t groups;        /* groups of E / groups neighbouring experts; 1 = none */
    int32_t top_groups;    /* groups whose experts may be selected */
    int32_t group_top;     /* a group's value: 1 its largest key, 2 the sum of its two largest score + bias */
    int32_t renormalize;   /* 1: weights divided by their sum over the k selected */
    float scale;           /* the weights' factor */
} moe_scoring;

/*
 * Each token's k experts and weights from its logits:
 *   s = scores(l); key = l without a bias (s is in the order of l), else s + bias;
 *   the top_groups groups of the largest values keep their experts;
 *   the k experts of the largest keys, descending;
 *   w = s of the selected, / their sum if renormalize, * scale.
 * Ties (of groups and of experts) go to the lower index. The order is that of real
 * arithmetic up to fp64's rounding, whatever the logits' type.
 * A logit of -inf is an expert with score 0 (selected, with weight 0, where no
 * other is left; a softmax of nothing but -inf is all 0, and so is the
 * renormalization of a sum of 0). A NaN logit comes after all others, and makes
 * its row's k weights NaN. A bias of +inf puts an expert before all others, one of -inf
 * behind them; several of them are ties.
 * Weights are fp32: within (56 + 2 d) 2^-24 of themselves, d the logit's distance from its
 * row's largest (sigmoid: 28 * 2^-24); scores below 2^-126 may be 0.
 * In:  logits[T,E] of type dtype, rows `stride` elements apart; scoring (null:
 *      softmax, no bias, no groups, not renormalized, scale 1).
 * Out: topk_idx[T,k], topk_w[T,k].
 * 1 <= k <= 8, E <= 256, groups <= 32 and a divisor of E, group_top <= E / groups,
 * k <= top_groups * (E / groups). Pointers aligned to their type.
 */
moe_status moe_route_logits(int64_t T, int32_t E, int32_t k, moe_dtype dtype, const void* logits, int64_t stride,
                            const moe_scoring* scoring, int32_t* topk_idx, float* topk_w, moe_stream_t stream);

/* relu: max(x, 0); silu: x / (1 + e^-x); gelu: x (1 + erf(x / sqrt 2)) / 2; gelu_tanh:
 * x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2. In fp32, before the output's rounding:
 * gelu within 2^-19 of itself (for 16-bit outputs 2^-15), silu and gelu_tanh within (5 + 3 |u|)
 * 2^-23, e^-u being their exponential (0 where that passes 2^126). */
typedef enum {
    MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3, MOE_ACT_GELU_TANH = 4
} moe_activation;

/* A weight's layout: [G,K,N] (as the bf16 entry points' weights) or [G,N,K]. */
typedef enum { MOE_WEIGHT_KN = 0, MOE_WEIGHT_NK = 1 } moe_weight_layout;

typedef struct {
    const void* bias;            /* [G,N], or null */
    moe_dtype bias_dtype;        /* fp32, or the operands' type */
    moe_activation activation;
    const void* residual;        /* [R,N] of the output's type, or null; may be the output's memory with its stride */
    int64_t residual_stride;     /* elements from row to row */
} moe_epilogue;

/* Bytes of moe_linear's workspace, for any sizes. Its first MOE_LINEAR_WORKSPACE_ZEROS
 * bytes have to be zero before its first use, and again after moe_check has returned
 * MOE_ERR_TIMEOUT for it; the calls leave them as the next call needs them. Two calls
 * that share a workspace must not overlap. */
#define MOE_LINEAR_WORKSPACE_ZEROS 2304
size_t moe_linear_workspace_size(void);

/*
 * Grouped product: out[p,:] = act(a[p,:] w[g] + bias[g]) + residual[p,:] for the rows
 * p of group g, offsets[g] <= p < offsets[g+1] (offsets null = one group of R
 * rows; G is then 1). Sums, bias, activation and residual in fp32, rounded once.
 * Rows outside [offsets[0], offsets[G]) are not written. Offsets that decrease or
 * leave [0, R] set MOE_ERR_DEVICE_BOUNDS in the device error word and nothing is
 * computed.
 * In:  a[R,K] of type dtype (bf16 or fp16), rows a_stride elements apart;
 *      offsets[G+1] (device); w of type dtype; epilogue (nullable).
 * Out: out[R,N] of type out_dtype (dtype or fp32), rows out_stride apart; its memory
 *      may be the residual's, and no other input's.
 * K a multiple of 8, for MOE_WEIGHT_KN N too, both up to 2^30; G <= 256; a and w 16-byte aligned, a_stride a multiple of 8,
 * the others aligned to their type.
 */
moe_status moe_linear(int64_t R, int32_t K, int32_t N, int32_t G, moe_dtype dtype, const void* a, int64_t a_stride,
                      const int32_t* offsets, const void* w, moe_weight_layout layout, const moe_epilogue* epilogue,
                      moe_dtype out_dtype, void* out, int64_t out_stride, void* ws, size_t ws_bytes,
                      moe_stream_t stream);

/* Test hook (host only): which kernel a product of these sizes runs on a device of
 * num_sms SMs: 0 tiles of up to 32 rows, 1 of up to 128 (one CTA per MMA), 2 and 3 a
 * CTA pair with up to 256 and 128; -1 for sizes that the call refuses (with MOE_WEIGHT_KN). The result does not depend on it but for
 * the order of its sums. */
int32_t moe_selftest_linear_form(int64_t R, int32_t K, int32_t N, int32_t G, int32_t num_sms);

/* Test hook (host only): the schedule of a product on a device of num_sms SMs, as its
 * kernel derives it from the offsets (offsets[G+1] on the host, null = one group): the first
 * `whole` tiles one a CTA (or pair), the K blocks of the others, end to end, in `segments`
 * equal runs, one a CTA. */
typedef struct {
    int32_t form;         /* moe_selftest_linear_form */
    int32_t units;        /* CTAs (or pairs) */
    int32_t tiles;
    int32_t whole;
    int32_t segments;     /* 0: no tile is cut */
    int32_t part_rows;    /* rows that a part of a cut tile has room for in the workspace */
    int32_t most_parts;   /* of a cut tile */
} moe_linear_schedule;
moe_status moe_selftest_linear_schedule(int64_t R, int32_t K, int32_t N, int32_t G, const int32_t* offsets,
                                        int32_t num_sms, moe_linear_schedule* schedule);

/*
 * The weighted sum of experts' rows, back in token order:
 *   out[t,:] = sum over ranks j (in order) of topk_w[t,j] y[inv_pos[t,j],:]
 *              + residual[t,:], in fp32, rounded once.
 * A rank whose inv_pos lies outside [0, R) (a dropped assignment: -1) adds nothing.
 * In:  y[R,H] of type dtype; inv_pos[T,k] (moe_permute's), topk_w[T,k]; residual[T,H]
 *      of type out_dtype (nullable; may be the output's memory with its stride).
 * Out: out[T,H] of type out_dtype.
 * 1 <= k <= 8; H a multiple of 8; y, residual and out 16-byte aligned with rows of
 * multiples of 16 bytes, their strides in elements.
 */
moe_status moe_combine_rows(int64_t T, int32_t H, int32_t k, int64_t R, moe_dtype dtype, const void* y,
                            int64_t y_stride, const int32_t* inv_pos, const float* topk_w, moe_dtype out_dtype,
                            const void* residual, int64_t residual_stride, void* out, int64_t out_stride,
                            moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
