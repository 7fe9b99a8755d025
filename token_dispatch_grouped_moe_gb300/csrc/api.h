// api.h -- what the files of the C ABI (api.cu, api_fp8.cu) share: host code
// only, internal to the library.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/moe.h"

namespace moe {

// An NVTX range over the host code that enqueues one stage: a profiler or
// tracer that records NVTX (ncu --nvtx, Nsight Systems) attributes each
// kernel to the stage that launched it ("moe/route", "moe/gemm0", ...). With
// no tool attached, a push/pop pair is a couple of branches (NVTX v3 is
// header-only and loads no library unless a tool asks for it).
struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    void next(const char* name)   // close this range and open the next stage's
    {
        nvtxRangePop();
        nvtxRangePushA(name);
    }
    Range(const Range&) = delete;
    Range& operator=(const Range&) = delete;
};

#define MOE_TRY(expr)                                  \
    do {                                               \
        cudaError_t e_ = (expr);                       \
        if (e_ != cudaSuccess) return MOE_ERR_CUDA;    \
    } while (0)

#define MOE_TRY_STATUS(expr)                           \
    do {                                               \
        moe_status s_ = (expr);                        \
        if (s_ != MOE_OK) return s_;                   \
    } while (0)

// SMs of the current device, or -1.
int num_sms_current();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// The status of a call whose launches returned e: with MOE_DEBUG=1 it
// synchronises and reads the error word at the start of ws (if any).
moe_status finish(cudaError_t e, void* ws, cudaStream_t s);

// The routing half of a layer call and the scratch of its other half, all in a
// workspace of moe_workspace_size(dims) bytes at `w`.
struct Routed {
    int32_t *topk_idx, *counts, *offsets, *src_row, *inv_pos, *tile_start;
    float* topk_w;
    unsigned char *x_perm, *h, *h_shared;   // [R, H], [R, F], [T, F_shared] of 2 bytes an element
    float* slot;                            // [k (+ 1 with a shared expert), T, H]
    float* shared_gate;                     // [T]
};
Routed routed_of(const moe_dims& d, const moe_routing_out* routing, unsigned char* w);
// Routes x and sorts the assignments by expert, by the per-shape table. The
// stage ranges are "moe/route" (open in `stage` at the call) and "moe/permute".
moe_status route_and_sort(const moe_dims& d, int router, const moe_bf16* x, const moe_bf16* Wg, const float* bias,
                          const moe_gating* gating, const Routed& r, unsigned char* w, uint32_t* err, int sms,
                          const moe_stage_events* events, Range& stage, cudaStream_t s);

}  // namespace moe
