"""Python binding of the C ABI in ``include/moe.h`` (ctypes).

Argument marshalling only: every step of the layer runs in the CUDA library.
Tensors are torch CUDA tensors (torch provides device memory and streams);
their data pointers and the current CUDA stream are passed through. If the
library has not been built, :func:`load` raises: there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_gb300.so")

MOE_OK = 0
MOE_ERR_TIMEOUT = 5
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_DEVICE_BOUNDS"}

EXPORTS = ["moe_version", "moe_status_string", "moe_workspace_size", "moe_check", "moe_route",
           "moe_permute", "moe_expert_ffn", "moe_combine", "moe_layer_forward", "moe_set_option",
           "moe_get_option", "moe_permute_static", "moe_route_ex", "moe_layer_forward_ex",
           "moe_layer_plan", "moe_selftest_wait_timeout", "moe_launch_count", "moe_selftest_route_tc",
           "moe_layer_forward_host", "moe_host_chunks", "moe_fp8_workspace_size", "moe_add_rmsnorm_fp8",
           "moe_fp8_quantize_weight", "moe_fp8_matmul", "moe_fp8_gated", "moe_fp8_layer_forward",
           "moe_selftest_fp8_form", "moe_route_logits", "moe_linear_workspace_size", "moe_linear", "moe_combine_rows",
           "moe_selftest_linear_form", "moe_selftest_linear_schedule", "moe_selftest_hold"]

OPT_GEMM0_A = 0
GEMM0_A_PERMUTED = 0      # dispatch copies token rows to x_perm; GEMM0 loads dense tiles
GEMM0_A_TMA_GATHER = 1    # GEMM0 producer gathers token rows with TMA gather4
GEMM0_A_CP_GATHER = 2     # a GEMM0 producer warp gathers token rows with cp.async
OPT_COMBINE = 1
COMBINE_AUTO = 0          # fused when the last GEMM1 has K >= 4096
COMBINE_FUSED = 1         # GEMM1's epilogue: the last contribution sums the slots
COMBINE_SEPARATE = 2      # a streaming combine kernel after the GEMMs
OPT_GEMM_FUSION = 2
GEMM_FUSION_AUTO = 0      # by shape (the library's table)
GEMM_FUSION_ON = 1        # both routed GEMMs in one persistent launch
GEMM_FUSION_OFF = 2       # two launches
OPT_CTA_GROUP = 3
CTA_GROUP_AUTO = 0        # by rows per expert (the library's table)
CTA_GROUP_ONE = 1         # one CTA per 128 x 256 MMA tile
CTA_GROUP_PAIR = 2        # a 2-CTA cluster per 256 x 256 MMA tile (tcgen05 cta_group::2)
OPT_X_PERM_COPY = 4
X_PERM_COPY_AUTO = 0      # by the library's table
X_PERM_COPY_INLINE = 1    # GEMM0's copy warps fill x_perm while the GEMM runs
X_PERM_COPY_KERNEL = 2    # a copy kernel before GEMM0
OPT_ROUTER = 5
ROUTER_OPT_AUTO = 0       # by the library's table
ROUTER_OPT_FMA = 1        # the FMA routers (the canonical order itself)
ROUTER_OPT_TENSOR = 2     # the tensor-core router wherever it applies


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("F", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("F_shared", ctypes.c_int32)]


class StageEvents(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("before_route", "before_permute", "before_gemm0",
                                               "before_gemm1", "before_shared", "before_combine",
                                               "after_combine")]


class Gating(ctypes.Structure):
    _fields_ = [("renormalize", ctypes.c_int32), ("shared_gate", ctypes.c_void_p)]


class RoutingOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_idx", "topk_w", "counts", "offsets", "src_row",
                                               "inv_pos")]


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("router", "gemm0_a", "combine", "gemm_fusion", "tile_m",
                                              "tile_n", "tile_k", "stages", "cta_group",
                                              "cta_group_gemm1", "x_perm_copy")]


class Scoring(ctypes.Structure):
    _fields_ = [("scores", ctypes.c_int32), ("bias", ctypes.c_void_p), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("bias_dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64)]


class LinearSchedule(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("form", "units", "tiles", "whole", "segments", "part_rows", "most_parts")]


class Fp8Ffn(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w1", "w1_scale", "w3", "w3_scale", "w2", "w2_scale")]


ROUTER_STREAM, ROUTER_SLICED, ROUTER_CLUSTER, ROUTER_BLOCK, ROUTER_TENSOR = 0, 1, 2, 3, 4


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (raises if it is missing: build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: run `python -m token_dispatch_grouped_moe_gb300.build`"
                           " (the MoE layer has no CPU fallback)")
    lib = ctypes.CDLL(path)
    P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(Dims)
    lib.moe_version.restype = ctypes.c_int
    lib.moe_version.argtypes = []
    lib.moe_launch_count.restype = ctypes.c_uint64
    lib.moe_launch_count.argtypes = []
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_workspace_size.restype = sz
    lib.moe_workspace_size.argtypes = [D]
    lib.moe_set_option.restype = ctypes.c_int
    lib.moe_set_option.argtypes = [ctypes.c_int, ctypes.c_int]
    lib.moe_get_option.restype = ctypes.c_int
    lib.moe_get_option.argtypes = [ctypes.c_int]
    lib.moe_check.restype = ctypes.c_int
    lib.moe_check.argtypes = [P, P]
    lib.moe_route.restype = ctypes.c_int
    lib.moe_route.argtypes = [D, P, P, P, P, P, P]
    lib.moe_permute.restype = ctypes.c_int
    lib.moe_permute.argtypes = [D, P, P, P, P, P, P, P, P, sz, P]
    lib.moe_permute_static.restype = ctypes.c_int
    lib.moe_permute_static.argtypes = [D, P, P, P, P, P, P, P, P]
    lib.moe_expert_ffn.restype = ctypes.c_int
    lib.moe_expert_ffn.argtypes = [D, P, P, P, P, P, P, P, P, P, sz, P]
    lib.moe_combine.restype = ctypes.c_int
    lib.moe_combine.argtypes = [D, P, i32, P, P]
    lib.moe_route_ex.restype = ctypes.c_int
    lib.moe_route_ex.argtypes = [D, P, P, P, ctypes.POINTER(Gating), P, P, P]
    lib.moe_layer_forward_ex.restype = ctypes.c_int
    lib.moe_layer_forward_ex.argtypes = [D, P, P, P, ctypes.POINTER(Gating), P, P, P, P, P, P, P,
                                         ctypes.POINTER(RoutingOut), P, sz, ctypes.POINTER(StageEvents), P]
    lib.moe_selftest_wait_timeout.restype = ctypes.c_int
    lib.moe_selftest_wait_timeout.argtypes = [i32, P]
    lib.moe_selftest_hold.restype = ctypes.c_int
    lib.moe_selftest_hold.argtypes = [i32, P]
    lib.moe_selftest_route_tc.restype = ctypes.c_int
    lib.moe_selftest_route_tc.argtypes = [D, P, P, P, i32, i32, P, P, P, P, ctypes.POINTER(ctypes.c_int64),
                                          P, sz, P]
    lib.moe_layer_plan.restype = ctypes.c_int
    lib.moe_layer_plan.argtypes = [D, ctypes.POINTER(Plan)]
    lib.moe_layer_forward.restype = ctypes.c_int
    lib.moe_layer_forward.argtypes = [D, P, P, P, P, P, P, P, P, P, P, ctypes.POINTER(RoutingOut), P,
                                      sz, ctypes.POINTER(StageEvents), P]
    lib.moe_layer_forward_host.restype = ctypes.c_int
    lib.moe_layer_forward_host.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, P, i32, P, sz, P]
    lib.moe_host_chunks.restype = i32
    lib.moe_host_chunks.argtypes = [D]
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.moe_fp8_workspace_size.restype = sz
    lib.moe_fp8_workspace_size.argtypes = [D]
    lib.moe_add_rmsnorm_fp8.restype = ctypes.c_int
    lib.moe_add_rmsnorm_fp8.argtypes = [i64, i32, i32, P, i64, P, i64, P, f32, P, i64, P, P, P, P]
    lib.moe_fp8_quantize_weight.restype = ctypes.c_int
    lib.moe_fp8_quantize_weight.argtypes = [i32, i32, i32, P, P, P, P]
    lib.moe_fp8_matmul.restype = ctypes.c_int
    lib.moe_fp8_matmul.argtypes = [i64, i32, i32, i32, P, P, P, P, P, i32, P, P, sz, P]
    lib.moe_fp8_gated.restype = ctypes.c_int
    lib.moe_fp8_gated.argtypes = [i64, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.moe_selftest_fp8_form.restype = i32
    lib.moe_selftest_fp8_form.argtypes = [i64, i32, i32, i32, i32, i32]
    lib.moe_fp8_layer_forward.restype = ctypes.c_int
    lib.moe_fp8_layer_forward.argtypes = [D, P, P, P, P, P, ctypes.POINTER(Gating), ctypes.POINTER(Fp8Ffn),
                                          ctypes.POINTER(Fp8Ffn), P, ctypes.POINTER(RoutingOut), P, sz, P]
    lib.moe_route_logits.restype = ctypes.c_int
    lib.moe_route_logits.argtypes = [i64, i32, i32, i32, P, i64, ctypes.POINTER(Scoring), P, P, P]
    lib.moe_linear_workspace_size.restype = sz
    lib.moe_linear_workspace_size.argtypes = []
    lib.moe_linear.restype = ctypes.c_int
    lib.moe_linear.argtypes = [i64, i32, i32, i32, i32, P, i64, P, P, i32, ctypes.POINTER(Epilogue), i32, P, i64, P, sz, P]
    lib.moe_selftest_linear_form.restype = i32
    lib.moe_selftest_linear_form.argtypes = [i64, i32, i32, i32, i32]
    lib.moe_selftest_linear_schedule.restype = ctypes.c_int
    lib.moe_selftest_linear_schedule.argtypes = [i64, i32, i32, i32, P, i32, ctypes.POINTER(LinearSchedule)]
    lib.moe_combine_rows.restype = ctypes.c_int
    lib.moe_combine_rows.argtypes = [i64, i32, i32, i64, i32, P, i64, P, P, i32, P, i64, P, i64, P]
    _lib = lib
    return lib


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _raw_stream() -> int:
    """The current stream's handle (torch.cuda.current_stream() makes an object
    around it: 2.8 us a call)."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _stream(stream=None):
    return ctypes.c_void_p(_raw_stream() if stream is None else stream.cuda_stream)


def _on(device, stream):
    """The context of a call: its tensors' device, and the stream given or that
    device's current one. What is allocated within is memory of that stream."""
    if device.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got tensors on {device}")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream: of {stream.device}, but the tensors are on {device}")
        return torch.cuda.stream(stream)
    if device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _ok(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def set_gemm0_a(mode: int) -> None:
    """Choose how GEMM0 obtains its token rows (GEMM0_A_PERMUTED or GEMM0_A_TMA_GATHER)."""
    _ok(load().moe_set_option(OPT_GEMM0_A, int(mode)), "moe_set_option")


def get_gemm0_a() -> int:
    return int(load().moe_get_option(OPT_GEMM0_A))


def set_combine(mode: int) -> None:
    """Choose where the layer sums the expert rows (COMBINE_AUTO / _FUSED / _SEPARATE)."""
    _ok(load().moe_set_option(OPT_COMBINE, int(mode)), "moe_set_option")


def get_combine() -> int:
    return int(load().moe_get_option(OPT_COMBINE))


def set_gemm_fusion(mode: int) -> None:
    """Run the routed GEMMs as one launch or two (GEMM_FUSION_AUTO / _ON / _OFF)."""
    _ok(load().moe_set_option(OPT_GEMM_FUSION, int(mode)), "moe_set_option")


def get_gemm_fusion() -> int:
    return int(load().moe_get_option(OPT_GEMM_FUSION))


def set_cta_group(mode: int) -> None:
    """CTAs per MMA of the dense-A expert GEMMs (CTA_GROUP_AUTO / _ONE / _PAIR)."""
    _ok(load().moe_set_option(OPT_CTA_GROUP, int(mode)), "moe_set_option")


def get_cta_group() -> int:
    return int(load().moe_get_option(OPT_CTA_GROUP))


def set_x_perm_copy(mode: int) -> None:
    """Who fills x_perm for GEMM0 (X_PERM_COPY_AUTO / _INLINE / _KERNEL)."""
    _ok(load().moe_set_option(OPT_X_PERM_COPY, int(mode)), "moe_set_option")


def get_x_perm_copy() -> int:
    return int(load().moe_get_option(OPT_X_PERM_COPY))


def set_router(mode: int) -> None:
    """Which router the layer call runs (ROUTER_OPT_AUTO / _FMA / _TENSOR)."""
    _ok(load().moe_set_option(OPT_ROUTER, int(mode)), "moe_set_option")


def route_tc_selftest(dims: Dims, x, Wg, ws, bias=None, renormalize=True, force_exact=False,
                      want_fast=False, stream=None):
    """The tensor-core router alone (test hook moe_selftest_route_tc).
    Returns (topk_idx, topk_w, fast_logits or None, fast_bound or None,
    number of tokens recomputed in the canonical order)."""
    T, k, E = dims.T, dims.k, dims.E
    dev = x.device
    with _on(dev, stream):
        idx = torch.empty(T, k, dtype=torch.int32, device=dev)
        w = torch.empty(T, k, dtype=torch.float32, device=dev)
        fast = torch.empty(T, E, dtype=torch.float32, device=dev) if want_fast else None
        bound = torch.empty(T, dtype=torch.float32, device=dev) if want_fast else None
        n = ctypes.c_int64(0)
        _ok(load().moe_selftest_route_tc(ctypes.byref(dims), _p(x), _p(Wg), _p(bias), int(renormalize),
                                         int(force_exact), _p(idx), _p(w), _p(fast), _p(bound),
                                         ctypes.byref(n), _p(ws), ws.numel(), _stream(stream)),
            "moe_selftest_route_tc")
        return idx, w, fast, bound, int(n.value)


def launch_count() -> int:
    """Kernels this library has launched in this process so far."""
    return int(load().moe_launch_count())


def selftest_wait_timeout(limit_ms: int = 200, stream=None) -> int:
    """Status of the bounded-wait self-test (MOE_ERR_TIMEOUT is the expected one)."""
    return int(load().moe_selftest_wait_timeout(int(limit_ms), _stream(stream)))


def selftest_hold(ms: int, stream=None) -> None:
    """Keeps the stream busy for ``ms`` with the next kernel resident beside it (test hook)."""
    _ok(load().moe_selftest_hold(int(ms), _stream(stream)), "moe_selftest_hold")


def layer_plan(dims: Dims) -> Plan:
    """The configuration moe_layer_forward runs for this shape (host only)."""
    p = Plan()
    _ok(load().moe_layer_plan(ctypes.byref(dims), ctypes.byref(p)), "moe_layer_plan")
    return p


def make_dims(T, H, F, E, k, F_shared=0) -> Dims:
    return Dims(int(T), int(H), int(F), int(E), int(k), int(F_shared))


def workspace_size(dims: Dims) -> int:
    return int(load().moe_workspace_size(ctypes.byref(dims)))


def workspace(dims: Dims, device=None) -> torch.Tensor:
    """A workspace (uint8) for ``dims``; its head, the error word, is zero."""
    n = workspace_size(dims)
    if n == 0:
        raise MoeError(1, "workspace_size")
    return _zero_headed(n, 256, device)


def _zero_headed(n: int, head: int, device) -> torch.Tensor:
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    ws[:head].zero_()
    return ws


def check(ws: torch.Tensor, stream=None) -> int:
    """Synchronise and return (and clear) the device error status in ``ws``."""
    with _on(ws.device, stream):
        return int(load().moe_check(_p(ws), _stream()))


def _gating(renormalize=True, shared_gate=None):
    if renormalize and shared_gate is None:
        return None
    return Gating(1 if renormalize else 0, None if shared_gate is None else shared_gate.data_ptr())


def route(dims: Dims, x, Wg, bias=None, topk_idx=None, topk_w=None, stream=None, renormalize=True):
    T, k = dims.T, dims.k
    dev = x.device
    with _on(dev, stream):
        topk_idx = topk_idx if topk_idx is not None else torch.empty(T, k, dtype=torch.int32, device=dev)
        topk_w = topk_w if topk_w is not None else torch.empty(T, k, dtype=torch.float32, device=dev)
        g = _gating(renormalize)
        _ok(load().moe_route_ex(ctypes.byref(dims), _p(x), _p(Wg), _p(bias),
                                ctypes.byref(g) if g is not None else None, _p(topk_idx), _p(topk_w),
                                _stream(stream)), "moe_route_ex")
        return topk_idx, topk_w


def _row_type(dims: Dims, x, dev):
    """The type of the rows that a dispatch copies: x's, bf16 or fp16 (16-bit values, as they are)."""
    if x is None:
        return torch.bfloat16
    # (T * H values and more in any shape: a batch of sequences, a longer buffer)
    if (x.dtype not in (torch.bfloat16, torch.float16) or x.numel() < dims.T * dims.H or not x.is_contiguous()
            or x.device != dev):
        raise ValueError(f"x: expected a contiguous bf16 or fp16 tensor of {dims.T} x {dims.H} values on {dev}, got "
                         f"{x.dtype} {tuple(x.shape)} (strides {x.stride()}) on {x.device}")
    return x.dtype


def permute(dims: Dims, topk_idx, ws, x=None, want_x_perm=False, stream=None):
    """The assignments sorted by expert: (counts [E], offsets [E+1], src_row [T*k],
    inv_pos [T*k], and with ``want_x_perm`` the rows of x [T,H], bf16 or fp16, in that
    order, else None)."""
    R, E = dims.T * dims.k, dims.E
    dev = topk_idx.device
    row_type = _row_type(dims, x, dev) if want_x_perm else None
    with _on(dev, stream):
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        src_row = torch.empty(R, dtype=torch.int32, device=dev)
        inv_pos = torch.empty(R, dtype=torch.int32, device=dev)
        x_perm = torch.empty(R, dims.H, dtype=row_type, device=dev) if want_x_perm else None
        _ok(load().moe_permute(ctypes.byref(dims), _p(topk_idx), _p(counts), _p(offsets), _p(src_row),
                               _p(inv_pos), _p(x), _p(x_perm), _p(ws), ws.numel(), _stream(stream)),
            "moe_permute")
        return counts, offsets, src_row, inv_pos, x_perm


def permute_static(dims: Dims, topk_idx, x=None, want_x_perm=False, stream=None):
    """Dispatch without a workspace (scratch is a fixed array inside the
    library; calls on one device must not overlap on the GPU)."""
    R, E = dims.T * dims.k, dims.E
    dev = topk_idx.device
    row_type = _row_type(dims, x, dev) if want_x_perm else None
    with _on(dev, stream):
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        src_row = torch.empty(R, dtype=torch.int32, device=dev)
        inv_pos = torch.empty(R, dtype=torch.int32, device=dev)
        x_perm = torch.empty(R, dims.H, dtype=row_type, device=dev) if want_x_perm else None
        _ok(load().moe_permute_static(ctypes.byref(dims), _p(topk_idx), _p(counts), _p(offsets),
                                      _p(src_row), _p(inv_pos), _p(x), _p(x_perm), _stream(stream)),
            "moe_permute_static")
        return counts, offsets, src_row, inv_pos, x_perm


def expert_ffn(dims: Dims, x, src_row, offsets, W1, W3, W2, topk_w, ws, slot=None, stream=None):
    with _on(x.device, stream):
        if slot is None:
            slot = torch.empty(dims.k, dims.T, dims.H, dtype=torch.float32, device=x.device)
        _ok(load().moe_expert_ffn(ctypes.byref(dims), _p(x), _p(src_row), _p(offsets), _p(W1), _p(W3),
                                  _p(W2), _p(topk_w), _p(slot), _p(ws), ws.numel(), _stream(stream)),
            "moe_expert_ffn")
        return slot


def combine(dims: Dims, slot, n_slots=None, out=None, stream=None):
    with _on(slot.device, stream):
        n_slots = n_slots if n_slots is not None else slot.shape[0]
        if out is None:
            out = torch.empty(dims.T, dims.H, dtype=torch.bfloat16, device=slot.device)
        _ok(load().moe_combine(ctypes.byref(dims), _p(slot), int(n_slots), _p(out), _stream(stream)),
            "moe_combine")
        return out


@dataclass
class Routing:
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    src_row: torch.Tensor
    inv_pos: torch.Tensor


def routing_buffers(dims: Dims, device) -> Routing:
    R = dims.T * dims.k
    i32 = dict(dtype=torch.int32, device=device)
    return Routing(torch.empty(dims.T, dims.k, **i32),
                   torch.empty(dims.T, dims.k, dtype=torch.float32, device=device),
                   torch.empty(dims.E, **i32), torch.empty(dims.E + 1, **i32),
                   torch.empty(R, **i32), torch.empty(R, **i32))


def layer_forward(dims: Dims, x, Wg, W1, W3, W2, ws, bias=None, W1s=None, W3s=None, W2s=None,
                  out=None, routing: Routing | None = None, events: StageEvents | None = None,
                  stream=None, renormalize=True, shared_gate=None):
    with _on(x.device, stream):
        if out is None:
            out = torch.empty(dims.T, dims.H, dtype=torch.bfloat16, device=x.device)
        r = None
        if routing is not None:
            r = RoutingOut(*(ctypes.c_void_p(getattr(routing, n).data_ptr()) for n in
                             ("topk_idx", "topk_w", "counts", "offsets", "src_row", "inv_pos")))
        g = _gating(renormalize, shared_gate)
        if g is None:
            _ok(load().moe_layer_forward(ctypes.byref(dims), _p(x), _p(Wg), _p(bias), _p(W1), _p(W3), _p(W2),
                                         _p(W1s), _p(W3s), _p(W2s), _p(out),
                                         ctypes.byref(r) if r is not None else None, _p(ws), ws.numel(),
                                         ctypes.byref(events) if events is not None else None,
                                         _stream(stream)), "moe_layer_forward")
        else:
            _ok(load().moe_layer_forward_ex(ctypes.byref(dims), _p(x), _p(Wg), _p(bias), ctypes.byref(g),
                                            _p(W1), _p(W3), _p(W2), _p(W1s), _p(W3s), _p(W2s), _p(out),
                                            ctypes.byref(r) if r is not None else None, _p(ws), ws.numel(),
                                            ctypes.byref(events) if events is not None else None,
                                            _stream(stream)), "moe_layer_forward_ex")
        return out


def layer_forward_host(dims: Dims, x_host, Wg, W1, W3, W2, ws, x_dev, out_dev, out_host=None, bias=None,
                       W1s=None, W3s=None, W2s=None, n_chunks=0, stream=None):
    """moe_layer_forward_host: x_host and out_host in (pinned) host memory,
    x_dev/out_dev device staging buffers of [T, H] bf16; the chunks' copies
    overlap the layer's kernels. Returns out_host (valid once the stream has
    been synchronized)."""
    with _on(x_dev.device, stream):
        if out_host is None:
            out_host = torch.empty(dims.T, dims.H, dtype=torch.bfloat16).pin_memory()
        _ok(load().moe_layer_forward_host(ctypes.byref(dims), _p(x_host), _p(Wg), _p(bias), _p(W1), _p(W3), _p(W2),
                                          _p(W1s), _p(W3s), _p(W2s), _p(out_host), _p(x_dev), _p(out_dev),
                                          int(n_chunks), _p(ws), ws.numel(), _stream(stream)),
            "moe_layer_forward_host")
        return out_host


def host_chunks(dims: Dims) -> int:
    return int(load().moe_host_chunks(ctypes.byref(dims)))


class _Layer:
    """What the layer objects share: their sizes and a workspace for each stream."""

    def dims(self, T) -> Dims:
        return make_dims(T, self.H, self.F, self.E, self.k, self.Fs)

    def workspace(self, T, stream=None):
        """A workspace for calls of up to T rows, or more, on ``stream`` (the current
        one). It is made on that stream, before the work that uses it, and goes
        back to that stream's memory behind it. It grows by a quarter at least, so
        a batch that gets longer row by row does not make a new one every time.
        A stream that is captured gets a new one with each call, which belongs to
        the graph: zeroed at every replay, and never given to anyone else while
        the graph lives, as a workspace kept here is once it has been outgrown."""
        with _on(self.Wg.device, stream):
            if torch.cuda.is_current_stream_capturing():
                return self._new_workspace(self.dims(T))
            key = _raw_stream()
            rows, ws = self._ws.get(key, (-1, None))
            if rows < T:
                rows, ws = max(T, rows + rows // 4), None
                self._ws.pop(key, None)   # its memory first, then the longer one's
                ws = self._new_workspace(self.dims(rows))
                self._ws[key] = (rows, ws)
        return ws


class MoELayer(_Layer):
    """Weights and a workspace on one device; ``forward(x)`` runs the layer."""

    def __init__(self, Wg, W1, W3, W2, k, bias=None, W1s=None, W3s=None, W2s=None):
        self.Wg, self.W1, self.W3, self.W2, self.k, self.bias = Wg, W1, W3, W2, int(k), bias
        self.W1s, self.W3s, self.W2s = W1s, W3s, W2s
        self.H, self.E = Wg.shape
        self.F = W1.shape[2]
        self.Fs = 0 if W1s is None else W1s.shape[1]
        self._ws = {}

    def _new_workspace(self, dims):
        return workspace(dims, device=self.Wg.device)

    def forward(self, x, out=None, routing=None, events=None, stream=None):
        T = x.shape[0]
        return layer_forward(self.dims(T), x, self.Wg, self.W1, self.W3, self.W2, self.workspace(T, stream),
                             self.bias, self.W1s, self.W3s, self.W2s, out=out, routing=routing,
                             events=events, stream=stream)


# ------------------------------------------------------------------ 8 bits --

FP8 = torch.float8_e4m3fn
FP8_BLOCK = 128   # values that share one scale
FP8_WORKSPACE_ZEROS = 2304   # bytes of a workspace that have to be zero before its first use


def _fp8_blocks(n: int) -> int:
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


def _expect(t, name, shape, dtype, device):
    """Argument check: a contiguous tensor of this shape and type on this device."""
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")


# The calls whose kernels take microseconds (the norm, the products, and the three
# of the last section)
# check their arguments, allocate and launch in C++ (csrc/torch_binding.cpp).
_binding = None


def _load_binding():
    global _binding
    load()
    try:
        from . import _binding as module
    except ImportError as e:
        raise RuntimeError(f"the Python binding is missing or was built for another PyTorch ({e}): run "
                           "`python -m token_dispatch_grouped_moe_gb300.build --force`") from e
    _binding = module
    return module


def _handle(stream, t):
    """The handle of a stream given to a call on the tensor t."""
    if stream is None:
        return None
    _on(t.device, stream)
    return stream.cuda_stream


def fp8_workspace_size(dims: Dims | None = None) -> int:
    return int(load().moe_fp8_workspace_size(None if dims is None else ctypes.byref(dims)))


def fp8_workspace(dims: Dims | None = None, device=None) -> torch.Tensor:
    """A workspace of :func:`fp8_matmul` and :func:`fp8_gated` (any sizes), or of
    :func:`fp8_layer_forward` for ``dims`` (or fewer rows), zeros where the calls
    need them."""
    n = fp8_workspace_size(dims)
    if n == 0:
        raise MoeError(1, "fp8_workspace_size")
    return _zero_headed(n, FP8_WORKSPACE_ZEROS, device)


def add_rmsnorm_fp8(x, weight=None, residual=None, eps=1e-6, want_y=True, sum_out=None, stream=None):
    """r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight for the rows of
    x [T,H] (bf16, fp16 or fp32; any row stride from H on), and y in e4m3 with a scale
    for each row's block of 128. Returns (r, y, q, scale): r is None without a
    residual (``sum_out`` gives its memory: x and residual are allowed), y None
    with ``want_y=False``."""
    r = (_binding or _load_binding()).add_rmsnorm_fp8(x, weight, residual, eps, want_y, sum_out, _handle(stream, x))
    if type(r) is int:
        raise MoeError(r, "moe_add_rmsnorm_fp8")
    return r


def fp8_quantize_weight(w, stream=None):
    """w [G,K,N] bf16 -> (q [G,N,K] e4m3, scale [G, ceil(N/128), ceil(K/128)]):
    a weight's layout for the 8-bit products, made once."""
    G, K, N = w.shape
    _expect(w, "w", (G, K, N), torch.bfloat16, w.device)
    with _on(w.device, stream):
        q = torch.empty(G, N, K, dtype=FP8, device=w.device)
        scale = torch.empty(G, _fp8_blocks(N), _fp8_blocks(K), dtype=torch.float32, device=w.device)
        _ok(load().moe_fp8_quantize_weight(G, K, N, w.data_ptr(), q.data_ptr(), scale.data_ptr(), _stream()),
            "moe_fp8_quantize_weight")
    return q, scale


def fp8_matmul(a, a_scale, w, w_scale, ws, offsets=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """out[p] = a[p] w[g]^T for the rows p of group g, offsets[g] <= p <
    offsets[g+1] (one group without offsets): a [R,K] and w [G,N,K] in e4m3
    with their block scales, out [R,N] bf16 or fp32. Rows outside every group
    are not written."""
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out_dtype: bf16 or fp32 expected, got {out_dtype}")
    r = (_binding or _load_binding()).fp8_matmul(a, a_scale, w, w_scale, ws, offsets, out_dtype is torch.bfloat16, out,
                                                 _handle(stream, a))
    if type(r) is int:
        raise MoeError(r, "moe_fp8_matmul")
    return r


def fp8_gated(a, a_scale, w1, w1_scale, w3, w3_scale, ws, offsets=None, stream=None):
    """h[p] = silu(a[p] w1[g]^T) * (a[p] w3[g]^T) for the rows of each group as
    in :func:`fp8_matmul`, quantized: (h [R,F] e4m3, scale [R, ceil(F/128)])."""
    r = (_binding or _load_binding()).fp8_gated(a, a_scale, w1, w1_scale, w3, w3_scale, ws, offsets, _handle(stream, a))
    if type(r) is int:
        raise MoeError(r, "moe_fp8_gated")
    return r


FP8_FORM_WIDE, FP8_FORM_NARROW, FP8_FORM_PAIR = 0, 1, 2


def fp8_form_selftest(R, K, N, G=1, gated=False, num_sms=152) -> int:
    """Which kernel a product of these sizes runs (test hook moe_selftest_fp8_form)."""
    return int(load().moe_selftest_fp8_form(R, K, N, G, int(gated), num_sms))


@dataclass
class Fp8Weights:
    """One expert set's 8-bit weights, from bf16 W1, W3 [E,H,F] and W2 [E,F,H]."""
    w1: torch.Tensor
    w1_scale: torch.Tensor
    w3: torch.Tensor
    w3_scale: torch.Tensor
    w2: torch.Tensor
    w2_scale: torch.Tensor

    @classmethod
    def from_bf16(cls, W1, W3, W2, stream=None) -> "Fp8Weights":
        return cls(*(t for w in (W1, W3, W2) for t in fp8_quantize_weight(w, stream=stream)))

    def _struct(self, E, H, F, device) -> Fp8Ffn:
        for n, (N, K) in {"w1": (F, H), "w3": (F, H), "w2": (H, F)}.items():
            _expect(getattr(self, n), n, (E, N, K), FP8, device)
            _expect(getattr(self, n + "_scale"), n + "_scale", (E, _fp8_blocks(N), _fp8_blocks(K)), torch.float32,
                    device)
        return Fp8Ffn(*(getattr(self, n).data_ptr() for n, _ in Fp8Ffn._fields_))


def fp8_layer_forward(dims: Dims, x, xq, xq_scale, Wg, routed: Fp8Weights, ws, bias=None,
                      shared: Fp8Weights | None = None, out=None, routing: Routing | None = None, renormalize=True,
                      shared_gate=None, stream=None):
    """The whole layer on 8-bit experts: the router reads x [T,H] (bf16), the
    experts xq, xq_scale (the same rows quantized: y, q, scale of
    :func:`add_rmsnorm_fp8`). ``ws`` from ``fp8_workspace(dims)``."""
    T, H, dev = dims.T, dims.H, x.device
    _expect(x, "x", (T, H), torch.bfloat16, dev)
    _expect(xq, "xq", (T, H), FP8, dev)
    _expect(xq_scale, "xq_scale", (T, _fp8_blocks(H)), torch.float32, dev)
    _expect(Wg, "Wg", (H, dims.E), torch.bfloat16, dev)
    if bias is not None:
        _expect(bias, "bias", (dims.E,), torch.float32, dev)
    if shared_gate is not None:
        _expect(shared_gate, "shared_gate", (H,), torch.bfloat16, dev)
    if out is not None:
        _expect(out, "out", (T, H), torch.bfloat16, dev)
    if dims.F_shared > 0 and shared is None:
        raise ValueError("shared: the shared expert's weights are needed when F_shared > 0")
    f = routed._struct(dims.E, H, dims.F, dev)
    fs = shared._struct(1, H, dims.F_shared, dev) if dims.F_shared > 0 else None
    if ws.dtype != torch.uint8 or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous uint8 tensor on {dev}, got {ws.dtype} (strides {ws.stride()}) on "
                         f"{ws.device}")
    r = None
    if routing is not None:
        R, E = T * dims.k, dims.E
        sizes = {"topk_idx": (T, dims.k), "topk_w": (T, dims.k), "counts": (E,), "offsets": (E + 1,), "src_row": (R,),
                 "inv_pos": (R,)}
        for n, size in sizes.items():
            _expect(getattr(routing, n), n, size, torch.float32 if n == "topk_w" else torch.int32, dev)
        r = RoutingOut(*(ctypes.c_void_p(getattr(routing, n).data_ptr()) for n in sizes))
    g = _gating(renormalize, shared_gate)
    with _on(dev, stream):
        if out is None:
            out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        _ok(load().moe_fp8_layer_forward(ctypes.byref(dims), _p(x), _p(xq), _p(xq_scale), _p(Wg), _p(bias),
                                         ctypes.byref(g) if g is not None else None, ctypes.byref(f),
                                         ctypes.byref(fs) if fs is not None else None, _p(out),
                                         ctypes.byref(r) if r is not None else None, _p(ws), ws.numel(),
                                         _stream()), "moe_fp8_layer_forward")
    return out


class MoEFp8Layer(_Layer):
    """A pre-norm expert layer of a residual stream, served in 8 bits: the
    residual's addition, the norm and its quantization, then the layer on
    weights quantized once from bf16 (on the stream current at that time).
    ``forward(x, residual)`` returns (the layer's output, the residual stream
    that the next layer adds it to); with ``stream`` it runs, and takes its
    memory, there, behind what the caller has that stream wait for."""

    def __init__(self, norm_weight, Wg, W1, W3, W2, k, bias=None, W1s=None, W3s=None, W2s=None, eps=1e-6):
        self.norm_weight, self.Wg, self.bias, self.k, self.eps = norm_weight, Wg, bias, int(k), eps
        self.H, self.E = Wg.shape
        self.F = W1.shape[2]
        self.Fs = 0 if W1s is None else W1s.shape[1]
        self.routed = Fp8Weights.from_bf16(W1, W3, W2)
        self.shared = None if W1s is None else Fp8Weights.from_bf16(W1s[None], W3s[None], W2s[None])
        self._ws = {}

    def _new_workspace(self, dims):
        return fp8_workspace(dims, device=self.Wg.device)

    def forward(self, x, residual=None, routing=None, stream=None):
        T = x.shape[0]
        r, y, q, scale = add_rmsnorm_fp8(x, self.norm_weight, residual=residual, eps=self.eps, stream=stream)
        out = fp8_layer_forward(self.dims(T), y, q, scale, self.Wg, self.routed, self.workspace(T, stream),
                                bias=self.bias, shared=self.shared, routing=routing, stream=stream)
        return out, x if residual is None else r


# ------------------------------- routing from logits, products with an epilogue --

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}   # moe_dtype
SCORES = {"softmax": 0, "sigmoid": 1}                               # moe_scores
ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # moe_activation
LINEAR_WORKSPACE_ZEROS = 2304   # bytes of a workspace that have to be zero before its first use


def _one_of(value, table, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name}: one of {', '.join(map(str, table))} expected, got {value!r}") from None


def route_logits(logits, k, scores="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=False,
                 scale=1.0, topk_idx=None, topk_w=None, stream=None):
    """Each token's k experts and weights from its logits [T,E] (bf16, fp16 or
    fp32; any row stride from E on): (topk_idx [T,k] int32, topk_w [T,k] fp32).

    s = softmax(logits) or sigmoid(logits) by ``scores``; the experts are those of
    the largest s + bias (``bias`` [E] fp32, of the selection only), descending,
    ties to the lower index. With ``groups`` > 1 only the experts of the
    ``top_groups`` groups (of E / groups neighbours) of the largest value are
    selected: a group's value is its largest s + bias, or with ``group_top=2`` the sum
    of its two largest. The weights are s of the selected, divided by their sum
    with ``renormalize``, times ``scale``. A logit of -inf is an expert with score 0; a NaN
    makes its row's weights NaN."""
    sigmoid = scores == "sigmoid" or (scores != "softmax" and _one_of(scores, SCORES, "scores"))
    r = (_binding or _load_binding()).route_logits(logits, k, sigmoid, bias, groups, top_groups, group_top, renormalize,
                                                   scale, topk_idx, topk_w,
                                                   None if stream is None else _handle(stream, logits))
    if type(r) is int:
        raise MoeError(r, "moe_route_logits")
    return r


def linear_workspace(device=None) -> torch.Tensor:
    """A workspace of :func:`linear` (any sizes), zeros where the calls need them."""
    return _zero_headed(int(load().moe_linear_workspace_size()), LINEAR_WORKSPACE_ZEROS, device)


def linear(a, w, ws, bias=None, activation=None, residual=None, offsets=None, out_dtype=None, out=None, stream=None):
    """out[p] = act(a[p] w[g] + bias[g]) + residual[p] for the rows p of group g,
    offsets[g] <= p < offsets[g+1] (one group without offsets): a [R,K] in bf16 or
    fp16 (any row stride that is a multiple of 8), w [G,K,N] of its type, contiguous
    (N then a multiple of 8, as K) or the transpose of a contiguous [G,N,K] (any N); bias
    [G,N] in fp32 or a's type;
    ``activation`` None, "relu", "silu", "gelu" or "gelu_tanh"; out and residual [R,N]
    (any row stride from N on) in a's type or, with ``out_dtype``, fp32. ``out`` may be
    the residual's memory. Rows outside every group are not written."""
    f32 = out_dtype is torch.float32
    if not f32 and out_dtype is not None and out_dtype is not a.dtype:
        raise ValueError(f"out_dtype: {a.dtype} or fp32 expected, got {out_dtype}")
    act = 0 if activation is None else _one_of(activation, ACTIVATIONS, "activation")
    r = (_binding or _load_binding()).linear(a, w, ws, bias, act, residual, offsets, f32, out,
                                             None if stream is None else _handle(stream, a))
    if type(r) is int:
        raise MoeError(r, "moe_linear")
    return r


LINEAR_FORM_FEW, LINEAR_FORM_ONE, LINEAR_FORM_PAIR, LINEAR_FORM_PAIR_HALF = 0, 1, 2, 3


def linear_form_selftest(R, K, N, G=1, num_sms=152) -> int:
    """Which kernel a product of these sizes runs (test hook moe_selftest_linear_form)."""
    return int(load().moe_selftest_linear_form(R, K, N, G, num_sms))


def linear_schedule_selftest(counts, K, N, num_sms=152) -> LinearSchedule:
    """The schedule of a product over groups of ``counts`` rows (test hook moe_selftest_linear_schedule)."""
    offsets = (ctypes.c_int32 * (len(counts) + 1))()
    for g, c in enumerate(counts):
        offsets[g + 1] = offsets[g] + c
    s = LinearSchedule()
    _ok(load().moe_selftest_linear_schedule(sum(counts), K, N, len(counts), offsets, num_sms, ctypes.byref(s)),
        "moe_selftest_linear_schedule")
    return s


def combine_rows(y, inv_pos, topk_w, residual=None, out_dtype=None, out=None, stream=None):
    """out[t] = sum_j topk_w[t,j] y[inv_pos[t,j]] + residual[t], ranks in order, in
    fp32: the experts' rows y [R,H] (bf16, fp16 or fp32, any row stride of
    multiples of 16 bytes) back in token order. inv_pos (T * k int32, as of
    :func:`permute`) outside [0, R) adds nothing; out and residual [T,H] are of
    ``out_dtype`` (y's by default), and may be the same memory."""
    code = -1 if out_dtype is None else _one_of(out_dtype, DTYPES, "out_dtype")
    r = (_binding or _load_binding()).combine_rows(y, inv_pos, topk_w, residual, code, out,
                                                   None if stream is None else _handle(stream, y))
    if type(r) is int:
        raise MoeError(r, "moe_combine_rows")
    return r
