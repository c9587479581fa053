"""ctypes binding of include/megamoe.h: argument marshalling only.

Every function takes torch tensors (device memory) or plain integers and
forwards raw pointers to the C ABI of libmegamoe.so; all work happens in the
HIP kernels.  If the library is missing this module raises -- there is no
fallback.
"""

from __future__ import annotations

import ctypes
import os

import torch

from . import _build

MM_A16W16, MM_A8W8_FP8, MM_A8W8_INT8, MM_MXFP8, MM_MXFP4 = 0, 1, 2, 3, 4
MM_OUT_BF16, MM_OUT_F32 = 0, 1
USECASE = {"bf16": MM_A16W16, "fp8": MM_A8W8_FP8, "int8": MM_A8W8_INT8, "mxfp8": MM_MXFP8, "mxfp4": MM_MXFP4}
KERNEL_IDS = 25
MM_ROUTER_SOFTMAX, MM_ROUTER_SIGMOID = 0, 1
SCORING = {"softmax": MM_ROUTER_SOFTMAX, "sigmoid": MM_ROUTER_SIGMOID}
MM_FEW_BF16, MM_FEW_FP8, MM_FEW_FP8_BLOCK = 0, 1, 2
OUT_DTYPE = {"bf16": MM_OUT_BF16, "f32": MM_OUT_F32, "fp32": MM_OUT_F32}
FEW_FORMAT = {"bf16": MM_FEW_BF16, "fp8": MM_FEW_FP8, "fp8_block": MM_FEW_FP8_BLOCK}
MM_ELEMENT_BF16, MM_ELEMENT_F16, MM_ELEMENT_F32, MM_ELEMENT_8BIT = 0, 1, 2, 3
ELEMENT = {torch.bfloat16: MM_ELEMENT_BF16, torch.float16: MM_ELEMENT_F16, torch.float32: MM_ELEMENT_F32,
           torch.int8: MM_ELEMENT_8BIT, torch.uint8: MM_ELEMENT_8BIT, torch.float8_e4m3fn: MM_ELEMENT_8BIT}
MM_DEVERR_BAD_EXPERT, MM_DEVERR_BARRIER_TIMEOUT, MM_DEVERR_BAD_OFFSETS = 1, 2, 4


class MMProblem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("intermediate_hidden", ctypes.c_int64),
        ("num_experts", ctypes.c_int64),
        ("num_topk", ctypes.c_int64),
        ("usecase", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("clamp_activation", ctypes.c_int32),
        ("activation_clamp", ctypes.c_float),
        ("num_shared_experts", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
    ]


class MMPlan(ctypes.Structure):
    _fields_ = [
        ("prob", MMProblem),
        ("block_m", ctypes.c_int32),
        ("tile_l1", ctypes.c_int32),
        ("tile_l2", ctypes.c_int32),
        ("gate_up_group", ctypes.c_int32),
        ("pool_rows", ctypes.c_int64),
        ("x_pool_bytes", ctypes.c_int64),
        ("a_pool_bytes", ctypes.c_int64),
        ("x_pool_scale_bytes", ctypes.c_int64),
        ("a_pool_scale_bytes", ctypes.c_int64),
        ("w1_bytes", ctypes.c_int64),
        ("w2_bytes", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64),
        ("fused_workspace_bytes", ctypes.c_int64),
        ("checksum", ctypes.c_uint64),
        ("reserved", ctypes.c_int64 * 8),
    ]


class MMRouterProblem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("num_experts", ctypes.c_int64),
        ("num_topk", ctypes.c_int64),
        ("scoring", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("route_scale", ctypes.c_float),
        ("reserved0", ctypes.c_int32),
    ]


class MMRouterPlan(ctypes.Structure):
    _fields_ = [
        ("prob", MMRouterProblem),
        ("workspace_bytes", ctypes.c_int64),
        ("checksum", ctypes.c_uint64),
        ("reserved", ctypes.c_int64 * 4),
    ]


class MMFewProblem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("intermediate_hidden", ctypes.c_int64),
        ("num_experts", ctypes.c_int64),
        ("num_topk", ctypes.c_int64),
        ("weight_format", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("clamp_activation", ctypes.c_int32),
        ("activation_clamp", ctypes.c_float),
        ("num_shared_experts", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
    ]


class MMFewPlan(ctypes.Structure):
    _fields_ = [
        ("prob", MMFewProblem),
        ("workspace_bytes", ctypes.c_int64),
        ("checksum", ctypes.c_uint64),
        ("reserved", ctypes.c_int64 * 4),
    ]


class MMBlockProblem(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("out_features", ctypes.c_int64),
        ("in_features", ctypes.c_int64),
        ("num_groups", ctypes.c_int64),
    ]


class MMBlockPlan(ctypes.Structure):
    _fields_ = [
        ("prob", MMBlockProblem),
        ("workspace_bytes", ctypes.c_int64),
        ("checksum", ctypes.c_uint64),
        ("reserved", ctypes.c_int64 * 4),
    ]


class MMSortProblem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("num_experts", ctypes.c_int64),
        ("num_topk", ctypes.c_int64),
        ("element", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
    ]


class MMSortPlan(ctypes.Structure):
    _fields_ = [
        ("prob", MMSortProblem),
        ("workspace_bytes", ctypes.c_int64),
        ("checksum", ctypes.c_uint64),
        ("reserved", ctypes.c_int64 * 4),
    ]


class MMInt8Problem(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("out_features", ctypes.c_int64),
        ("in_features", ctypes.c_int64),
        ("num_groups", ctypes.c_int64),
        ("x_element", ctypes.c_int32),
        ("y_element", ctypes.c_int32),
    ]


class MMInt8Plan(ctypes.Structure):
    _fields_ = [
        ("prob", MMInt8Problem),
        ("workspace_bytes", ctypes.c_int64),
        ("dense_workspace_bytes", ctypes.c_int64),
        ("checksum", ctypes.c_uint64),
        ("reserved", ctypes.c_int64 * 4),
    ]


EXPORTS = [
    "mm_plan_create", "mm_prepare_weights", "mm_dispatch_layout", "mm_grouped_l1_swiglu",
    "mm_grouped_l2_combine", "mega_moe", "mega_moe_noalloc", "mm_read_device_error", "mm_debug_raw_accumulators",
    "mm_debug_fused_layout", "mm_read_kernel_clock", "mm_trace_enable", "mm_trace_collect", "mm_kernel_name", "mm_status_string",
    "mm_router_plan_create", "mm_router", "mm_few_plan_create", "mm_moe_few", "mm_block_quantize",
    "mm_block_plan_create", "mm_block_gemm", "mm_block_linear",
    "mm_sort_plan_create", "mm_sort_tokens", "mm_sort_rows", "mm_combine_tokens", "mm_combine_backward",
    "mm_swiglu", "mm_swiglu_backward",
    "mm_int8_quantize", "mm_int8_plan_create", "mm_int8_gemm", "mm_int8_linear",
]

_lib = None


class MMError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


def lib_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"HIP library not built: {path} missing (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i32p, f32p, u64 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64
    P = ctypes.POINTER(MMPlan)
    lib.mm_plan_create.argtypes = [ctypes.POINTER(MMProblem), P]
    lib.mm_prepare_weights.argtypes = [P, vp, vp, vp, vp, vp]
    lib.mm_dispatch_layout.argtypes = [P, i32p, vp, vp, i32p, i32p, i32p, i32p, vp, f32p, vp, u64, vp]
    lib.mm_grouped_l1_swiglu.argtypes = [P, i32p, i32p, vp, f32p, vp, f32p, vp, f32p, vp, u64, vp]
    lib.mm_grouped_l2_combine.argtypes = [P, i32p, i32p, i32p, i32p, vp, f32p, vp, f32p, f32p, vp, vp, u64, vp]
    lib.mega_moe.argtypes = [P, vp, i32p, f32p, vp, vp, f32p, vp, f32p, vp, i32p, vp, u64, vp]
    lib.mega_moe_noalloc.argtypes = [P, vp, i32p, f32p, vp, vp, f32p, vp, f32p, vp, i32p, vp]
    lib.mm_read_device_error.argtypes = [P, vp, ctypes.POINTER(ctypes.c_int32), vp]
    lib.mm_debug_raw_accumulators.argtypes = [P, ctypes.c_int, i32p, i32p, vp, vp, i32p, vp, u64, vp]
    lib.mm_debug_fused_layout.argtypes = [P, vp, i32p, i32p, i32p, vp]
    lib.mm_read_kernel_clock.argtypes = [P, vp, ctypes.POINTER(ctypes.c_uint64), vp]
    RP, FP, BP = ctypes.POINTER(MMRouterPlan), ctypes.POINTER(MMFewPlan), ctypes.POINTER(MMBlockPlan)
    i64 = ctypes.c_int64
    lib.mm_router_plan_create.argtypes = [ctypes.POINTER(MMRouterProblem), RP]
    lib.mm_router.argtypes = [RP, vp, vp, f32p, vp, i32p, f32p, vp, u64, vp]
    lib.mm_few_plan_create.argtypes = [ctypes.POINTER(MMFewProblem), FP]
    lib.mm_moe_few.argtypes = [FP, vp, i32p, f32p, vp, vp, f32p, vp, f32p, vp, vp, u64, vp]
    lib.mm_block_quantize.argtypes = [i64, i64, vp, vp, f32p, vp]
    lib.mm_block_plan_create.argtypes = [ctypes.POINTER(MMBlockProblem), BP]
    lib.mm_block_gemm.argtypes = [BP, vp, f32p, vp, f32p, i32p, i32p, vp, vp]
    lib.mm_block_linear.argtypes = [BP, vp, vp, f32p, i32p, i32p, vp, vp, u64, vp]
    SP = ctypes.POINTER(MMSortPlan)
    lib.mm_sort_plan_create.argtypes = [ctypes.POINTER(MMSortProblem), SP]
    lib.mm_sort_tokens.argtypes = [SP, i32p, vp, vp, i32p, i32p, i32p, i32p, vp, vp, u64, vp]
    lib.mm_sort_rows.argtypes = [SP, vp, i32p, i32p, vp, vp]
    lib.mm_combine_tokens.argtypes = [SP, vp, i32p, f32p, vp, vp]
    lib.mm_combine_backward.argtypes = [SP, vp, vp, i32p, i32p, f32p, vp, f32p, vp]
    i32, f32 = ctypes.c_int32, ctypes.c_float
    lib.mm_swiglu.argtypes = [i64, i64, i32, i32, vp, i32, f32, vp, vp, f32p, vp]
    lib.mm_swiglu_backward.argtypes = [i64, i64, i32, i32, vp, vp, f32p, i32, f32, vp, vp]
    IP = ctypes.POINTER(MMInt8Plan)
    lib.mm_int8_quantize.argtypes = [i64, i64, i32, vp, vp, f32p, vp]
    lib.mm_int8_plan_create.argtypes = [ctypes.POINTER(MMInt8Problem), IP]
    lib.mm_int8_gemm.argtypes = [IP, vp, f32p, vp, f32p, i32p, i32p, vp, vp]
    lib.mm_int8_linear.argtypes = [IP, vp, vp, f32p, i32p, i32p, vp, vp, u64, vp]
    lib.mm_trace_enable.argtypes = [ctypes.c_int]
    lib.mm_trace_collect.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_double)]
    lib.mm_kernel_name.argtypes = [ctypes.c_int]
    lib.mm_kernel_name.restype = ctypes.c_char_p
    lib.mm_status_string.argtypes = [ctypes.c_int]
    lib.mm_status_string.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name not in ("mm_kernel_name", "mm_status_string"):
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().mm_status_string(status).decode()


def _ptr(t):
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if isinstance(stream, int):
        return stream
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream


def _check(fn, st):
    if st != 0:
        raise MMError(fn, st)


# ------------------------------------------------------------------ entries

def mm_plan_create(T, H, I, E, K, usecase="bf16", y_dtype="bf16", activation_clamp=None,
                   num_shared_experts=0) -> MMPlan:
    """activation_clamp: None (no clamp) or c >= 0 (H clamped to [-c, c] before SwiGLU);
    num_shared_experts: 0 or 1 (expert index E of the weight arrays)."""
    prob = MMProblem(T, H, I, E, K, USECASE.get(usecase, usecase) if isinstance(usecase, str) else usecase,
                     MM_OUT_F32 if y_dtype in ("f32", "fp32", MM_OUT_F32) else MM_OUT_BF16,
                     0 if activation_clamp is None else 1, 0.0 if activation_clamp is None else float(activation_clamp),
                     int(num_shared_experts), 0)
    plan = MMPlan()
    _check("mm_plan_create", load().mm_plan_create(ctypes.byref(prob), ctypes.byref(plan)))
    return plan


def mm_prepare_weights(plan, w1, w2, w1_out, w2_out, stream=None):
    _check("mm_prepare_weights", load().mm_prepare_weights(
        ctypes.byref(plan), _ptr(w1), _ptr(w2), _ptr(w1_out), _ptr(w2_out), _stream(stream)))


def mm_dispatch_layout(plan, topk_ids, x_active_mask, x, expert_counts, expert_offsets, pool_src, route_to_pool,
                       x_pool, x_pool_scale, workspace, stream=None):
    _check("mm_dispatch_layout", load().mm_dispatch_layout(
        ctypes.byref(plan), _ptr(topk_ids), _ptr(x_active_mask), _ptr(x), _ptr(expert_counts), _ptr(expert_offsets),
        _ptr(pool_src), _ptr(route_to_pool), _ptr(x_pool), _ptr(x_pool_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def mm_grouped_l1_swiglu(plan, expert_offsets, expert_counts, x_pool, x_pool_scale, w1, w1_scale,
                         a_pool, a_pool_scale, workspace, stream=None):
    _check("mm_grouped_l1_swiglu", load().mm_grouped_l1_swiglu(
        ctypes.byref(plan), _ptr(expert_offsets), _ptr(expert_counts), _ptr(x_pool), _ptr(x_pool_scale),
        _ptr(w1), _ptr(w1_scale), _ptr(a_pool), _ptr(a_pool_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def mm_grouped_l2_combine(plan, expert_offsets, expert_counts, pool_src, route_to_pool, a_pool,
                          a_pool_scale, w2, w2_scale, topk_weights, y, workspace, stream=None):
    _check("mm_grouped_l2_combine", load().mm_grouped_l2_combine(
        ctypes.byref(plan), _ptr(expert_offsets), _ptr(expert_counts), _ptr(pool_src), _ptr(route_to_pool),
        _ptr(a_pool), _ptr(a_pool_scale), _ptr(w2), _ptr(w2_scale), _ptr(topk_weights), _ptr(y),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def mega_moe(plan, x, topk_ids, topk_weights, x_active_mask, w1, w1_scale, w2, w2_scale, y, expert_token_nums,
             workspace, stream=None):
    _check("mega_moe", load().mega_moe(
        ctypes.byref(plan), _ptr(x), _ptr(topk_ids), _ptr(topk_weights), _ptr(x_active_mask), _ptr(w1), _ptr(w1_scale),
        _ptr(w2), _ptr(w2_scale), _ptr(y), _ptr(expert_token_nums), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def mega_moe_noalloc(plan, x, topk_ids, topk_weights, x_active_mask, w1, w1_scale, w2, w2_scale, y,
                     expert_token_nums, stream=None):
    _check("mega_moe_noalloc", load().mega_moe_noalloc(
        ctypes.byref(plan), _ptr(x), _ptr(topk_ids), _ptr(topk_weights), _ptr(x_active_mask), _ptr(w1),
        _ptr(w1_scale), _ptr(w2), _ptr(w2_scale), _ptr(y), _ptr(expert_token_nums), _stream(stream)))


def mm_router_plan_create(T, H, E, K, scoring="softmax", renormalize=True, route_scale=1.0) -> MMRouterPlan:
    sc = SCORING[scoring] if isinstance(scoring, str) else scoring
    prob = MMRouterProblem(T, H, E, K, sc, int(renormalize), route_scale, 0)
    plan = MMRouterPlan()
    _check("mm_router_plan_create", load().mm_router_plan_create(ctypes.byref(prob), ctypes.byref(plan)))
    return plan


def mm_router(plan, x, weight, bias, x_active_mask, topk_ids, topk_weights, workspace, stream=None):
    _check("mm_router", load().mm_router(
        ctypes.byref(plan), _ptr(x), _ptr(weight), _ptr(bias), _ptr(x_active_mask), _ptr(topk_ids),
        _ptr(topk_weights), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def mm_few_plan_create(T, H, I, E, K, weight_format="bf16", y_dtype="bf16", activation_clamp=None,
                       num_shared_experts=0) -> MMFewPlan:
    fmt = FEW_FORMAT[weight_format] if isinstance(weight_format, str) else weight_format
    yd = OUT_DTYPE.get(y_dtype, -1) if isinstance(y_dtype, str) else y_dtype      # -1: refused by the plan
    prob = MMFewProblem(T, H, I, E, K, fmt, yd, 0 if activation_clamp is None else 1,
                        0.0 if activation_clamp is None else activation_clamp, num_shared_experts, 0)
    plan = MMFewPlan()
    _check("mm_few_plan_create", load().mm_few_plan_create(ctypes.byref(prob), ctypes.byref(plan)))
    return plan


def mm_moe_few(plan, x, topk_ids, topk_weights, x_active_mask, w1, w1_scale, w2, w2_scale, y, workspace, stream=None):
    _check("mm_moe_few", load().mm_moe_few(
        ctypes.byref(plan), _ptr(x), _ptr(topk_ids), _ptr(topk_weights), _ptr(x_active_mask), _ptr(w1),
        _ptr(w1_scale), _ptr(w2), _ptr(w2_scale), _ptr(y), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def mm_block_quantize(rows, cols, x, codes, scales, stream=None):
    _check("mm_block_quantize", load().mm_block_quantize(rows, cols, _ptr(x), _ptr(codes), _ptr(scales),
                                                         _stream(stream)))


def mm_block_plan_create(M, N, K, G=1) -> MMBlockPlan:
    prob = MMBlockProblem(M, N, K, G)
    plan = MMBlockPlan()
    _check("mm_block_plan_create", load().mm_block_plan_create(ctypes.byref(prob), ctypes.byref(plan)))
    return plan


def mm_block_gemm(plan, a, a_scale, b, b_scale, group_offsets, group_counts, y, stream=None):
    _check("mm_block_gemm", load().mm_block_gemm(
        ctypes.byref(plan), _ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale), _ptr(group_offsets), _ptr(group_counts),
        _ptr(y), _stream(stream)))


def mm_block_linear(plan, x, b, b_scale, group_offsets, group_counts, y, workspace, stream=None):
    _check("mm_block_linear", load().mm_block_linear(
        ctypes.byref(plan), _ptr(x), _ptr(b), _ptr(b_scale), _ptr(group_offsets), _ptr(group_counts), _ptr(y),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def mm_sort_plan_create(T, H, E, K, element) -> MMSortPlan:
    prob = MMSortProblem(T, H, E, K, element, 0)
    plan = MMSortPlan()
    _check("mm_sort_plan_create", load().mm_sort_plan_create(ctypes.byref(prob), ctypes.byref(plan)))
    return plan


def mm_sort_tokens(plan, topk_ids, x_active_mask, x, counts, offsets, row_of_route, route_of_row, rows, workspace,
                   stream=None):
    _check("mm_sort_tokens", load().mm_sort_tokens(
        ctypes.byref(plan), _ptr(topk_ids), _ptr(x_active_mask), _ptr(x), _ptr(counts), _ptr(offsets),
        _ptr(row_of_route), _ptr(route_of_row), _ptr(rows), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)))


def mm_sort_rows(plan, x, offsets, row_of_route, rows, stream=None):
    _check("mm_sort_rows", load().mm_sort_rows(
        ctypes.byref(plan), _ptr(x), _ptr(offsets), _ptr(row_of_route), _ptr(rows), _stream(stream)))


def mm_combine_tokens(plan, rows, row_of_route, weights, y, stream=None):
    _check("mm_combine_tokens", load().mm_combine_tokens(
        ctypes.byref(plan), _ptr(rows), _ptr(row_of_route), _ptr(weights), _ptr(y), _stream(stream)))


def mm_combine_backward(plan, dy, rows, offsets, row_of_route, weights, drows, dweights, stream=None):
    _check("mm_combine_backward", load().mm_combine_backward(
        ctypes.byref(plan), _ptr(dy), _ptr(rows), _ptr(offsets), _ptr(row_of_route), _ptr(weights), _ptr(drows),
        _ptr(dweights), _stream(stream)))


def _clamp(activation_clamp):
    return (0, 0.0) if activation_clamp is None else (1, activation_clamp)


def mm_swiglu(rows, cols, element, gate_up_group, h, activation_clamp, a, codes, scales, stream=None):
    _check("mm_swiglu", load().mm_swiglu(rows, cols, element, gate_up_group, _ptr(h), *_clamp(activation_clamp), _ptr(a),
                                         _ptr(codes), _ptr(scales), _stream(stream)))


def mm_swiglu_backward(rows, cols, element, gate_up_group, da, codes, scales, activation_clamp, dh, stream=None):
    _check("mm_swiglu_backward", load().mm_swiglu_backward(
        rows, cols, element, gate_up_group, _ptr(da), _ptr(codes), _ptr(scales), *_clamp(activation_clamp), _ptr(dh),
        _stream(stream)))


def mm_int8_quantize(rows, cols, element, x, codes, scales, stream=None):
    _check("mm_int8_quantize", load().mm_int8_quantize(rows, cols, element, _ptr(x), _ptr(codes), _ptr(scales),
                                                       _stream(stream)))


def mm_int8_plan_create(M, N, K, G=1, x_element=MM_ELEMENT_BF16, y_element=MM_ELEMENT_BF16) -> MMInt8Plan:
    prob = MMInt8Problem(M, N, K, G, x_element, y_element)
    plan = MMInt8Plan()
    _check("mm_int8_plan_create", load().mm_int8_plan_create(ctypes.byref(prob), ctypes.byref(plan)))
    return plan


def mm_int8_gemm(plan, a, a_scale, b, b_scale, group_offsets, group_counts, y, stream=None):
    _check("mm_int8_gemm", load().mm_int8_gemm(
        ctypes.byref(plan), _ptr(a), _ptr(a_scale), _ptr(b), _ptr(b_scale), _ptr(group_offsets), _ptr(group_counts),
        _ptr(y), _stream(stream)))


def mm_int8_linear(plan, x, b, b_scale, group_offsets, group_counts, y, workspace, stream=None):
    _check("mm_int8_linear", load().mm_int8_linear(
        ctypes.byref(plan), _ptr(x), _ptr(b), _ptr(b_scale), _ptr(group_offsets), _ptr(group_counts), _ptr(y),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)))


def mm_read_device_error(plan, workspace, stream=None) -> int:
    """The device error word (mm_device_error bits) of the last call on `workspace`."""
    out = ctypes.c_int32(0)
    _check("mm_read_device_error", load().mm_read_device_error(
        ctypes.byref(plan), _ptr(workspace), ctypes.byref(out), _stream(stream)))
    torch.cuda.synchronize()
    return out.value


def mm_read_kernel_clock(plan, workspace, stream=None):
    """(shader clocks, 100 MHz ticks) spanned by workgroup 0 of the last mega_moe call; waits for the device."""
    out = (ctypes.c_uint64 * 4)()
    _check("mm_read_kernel_clock", load().mm_read_kernel_clock(ctypes.byref(plan), _ptr(workspace), out,
                                                                _stream(stream)))
    torch.cuda.synchronize()
    return out[1] - out[0], out[3] - out[2]


def mm_debug_raw_accumulators(plan, which, expert_offsets, expert_counts, act_pool, w_prepared, c_out,
                              workspace, stream=None):
    _check("mm_debug_raw_accumulators", load().mm_debug_raw_accumulators(
        ctypes.byref(plan), which, _ptr(expert_offsets), _ptr(expert_counts), _ptr(act_pool),
        _ptr(w_prepared), _ptr(c_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def mm_debug_fused_layout(plan, workspace, offsets_out, pool_src_out, route_to_pool_out, stream=None):
    _check("mm_debug_fused_layout", load().mm_debug_fused_layout(
        ctypes.byref(plan), _ptr(workspace), _ptr(offsets_out), _ptr(pool_src_out), _ptr(route_to_pool_out),
        _stream(stream)))


def mm_trace_enable(on: bool):
    _check("mm_trace_enable", load().mm_trace_enable(1 if on else 0))


def mm_trace_collect():
    """Returns {kernel name: (launches, total ms)} and clears the record."""
    n = (ctypes.c_int32 * KERNEL_IDS)()
    ms = (ctypes.c_double * KERNEL_IDS)()
    _check("mm_trace_collect", load().mm_trace_collect(n, ms))
    names = [load().mm_kernel_name(i).decode() for i in range(KERNEL_IDS)]
    return {name: (n[i], ms[i]) for i, name in enumerate(names) if name != "unknown"}


def mm_kernel_name(i: int) -> str:
    return load().mm_kernel_name(i).decode()
