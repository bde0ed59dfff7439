"""Sparse top-k Mixture-of-Experts feed-forward layer for AMD MI355X (gfx950).

Thin Python binding of libmoe.so (C ABI in include/moe.h).  The functions
below carry the C names and only marshal arguments: torch tensors supply
device pointers and the current HIP stream, every step of the layer runs in
the library's HIP kernels.  There is no CPU or fallback path: if libmoe.so
is missing, every call raises.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import (MOE_BF16, MOE_CALL_DOWN, MOE_CALL_FORWARD, MOE_CALL_GATE_UP,
                   MOE_CALL_PERMUTE, MOE_CALL_ROUTE, MOE_DROPLESS, MOE_F32, MOE_FP8_E4M3, MOE_MXFP4,
                   MOE_NOALLOC_SCRATCH_BYTES, MOE_OVERFLOW_DROP, MOE_OVERFLOW_NEXT_BEST, MoeShape,
                   MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU,
                   MOE_CALL_LINEAR, MOE_CALL_LINEAR_BACKWARD, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX,
                   MoeLinear, MoeRouter)

__all__ = ["MoEError", "MoeShape", "make_shape", "moe_status_string", "moe_version",
           "moe_workspace_bytes", "moe_route_topk", "moe_permute", "moe_expert_gemm_gate_up",
           "moe_expert_gemm_down", "moe_combine", "moe_forward", "moe_forward_noalloc",
           "MOE_NOALLOC_SCRATCH_BYTES", "MOE_F32", "MOE_BF16",
           "MOE_FP8_E4M3", "MOE_MXFP4", "MOE_DROPLESS", "MOE_CALL_PERMUTE", "MOE_CALL_GATE_UP",
           "MOE_CALL_DOWN", "MOE_CALL_FORWARD", "MOE_CALL_ROUTE", "MOE_OVERFLOW_DROP", "MOE_OVERFLOW_NEXT_BEST",
           "MoeRouter", "MoeLinear", "make_router", "make_linear", "moe_route_scored",
           "moe_route_scored_backward", "moe_combine_backward", "moe_forward_routed", "moe_linear",
           "moe_linear_backward", "moe_linear_workspace_bytes", "MOE_CALL_LINEAR",
           "MOE_CALL_LINEAR_BACKWARD", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "MOE_ACT_NONE",
           "MOE_ACT_RELU", "MOE_ACT_SILU", "MOE_ACT_GELU", "MOE_ACT_GELU_TANH"]

_DT = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8_e4m3": MOE_FP8_E4M3, "mxfp4": MOE_MXFP4}
_SCORE = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_ACT = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU,
        "gelu_tanh": MOE_ACT_GELU_TANH}
_OVF = {"drop": MOE_OVERFLOW_DROP, "next_best": MOE_OVERFLOW_NEXT_BEST}


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {moe_status_string(status)} ({status})")


def make_shape(T: int, d_model: int, d_ff: int, n_experts: int = 8, top_k: int = 2,
               capacity: int = MOE_DROPLESS, act_dtype="bf16", w_dtype="bf16",
               overflow="drop", n_shared: int = 0) -> MoeShape:
    a = _DT.get(act_dtype, act_dtype)
    w = _DT.get(w_dtype, w_dtype)
    return MoeShape(T, d_model, d_ff, n_experts, top_k, capacity, a, w, _OVF.get(overflow, overflow),
                    n_shared)


def shape_of(cfg) -> MoeShape:
    """Shape of a synthetic.MoEConfig."""
    return make_shape(cfg.T, cfg.d_model, cfg.d_ff, cfg.n_experts, cfg.top_k, cfg.capacity,
                      cfg.act_dtype, cfg.w_dtype, cfg.overflow, cfg.n_shared)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)
    if t.device.type != "cuda":
        raise ValueError("MoE tensors must live in device memory")
    if not t.is_contiguous():
        raise ValueError("MoE tensors must be contiguous (row-major)")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        if not torch.cuda.is_available():
            return None
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, status: int):
    if status != 0:
        raise MoEError(fn, status)


def moe_status_string(status: int) -> str:
    return _lib.load().moe_status_string(status).decode()


def moe_version() -> str:
    return _lib.load().moe_version().decode()


def moe_workspace_bytes(shape: MoeShape, call: int = MOE_CALL_FORWARD) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_workspace_bytes", _lib.load().moe_workspace_bytes(ctypes.byref(shape), call,
                                                                  ctypes.byref(n)))
    return n.value


def moe_route_topk(shape, x, w_gate, router_bias, topk_ids, topk_weights, logits=None,
                   next_ids=None, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("moe_route_topk", _lib.load().moe_route_topk(
        ctypes.byref(shape), _p(x), _p(w_gate), _p(router_bias), _p(topk_ids), _p(topk_weights),
        _p(logits), _p(next_ids), _p(workspace), ws_bytes, _stream(stream)))


def moe_permute(shape, topk_ids, topk_weights, next_ids, x, expert_counts, expert_offsets,
                perm_src, slot_to_row, drop_mask, x_perm, x_perm_scale=None, workspace=None,
                stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("moe_permute", _lib.load().moe_permute(
        ctypes.byref(shape), _p(topk_ids), _p(topk_weights), _p(next_ids), _p(x), _p(expert_counts),
        _p(expert_offsets), _p(perm_src), _p(slot_to_row), _p(drop_mask), _p(x_perm),
        _p(x_perm_scale), _p(workspace), ws_bytes, _stream(stream)))


def moe_expert_gemm_gate_up(shape, x_perm, x_perm_scale, expert_offsets, w1, w3, w1_scale,
                            w3_scale, h, h_scale=None, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("moe_expert_gemm_gate_up", _lib.load().moe_expert_gemm_gate_up(
        ctypes.byref(shape), _p(x_perm), _p(x_perm_scale), _p(expert_offsets), _p(w1), _p(w3),
        _p(w1_scale), _p(w3_scale), _p(h), _p(h_scale), _p(workspace), ws_bytes,
        _stream(stream)))


def moe_expert_gemm_down(shape, h, h_scale, expert_offsets, w2, w2_scale, y_perm,
                         workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("moe_expert_gemm_down", _lib.load().moe_expert_gemm_down(
        ctypes.byref(shape), _p(h), _p(h_scale), _p(expert_offsets), _p(w2), _p(w2_scale),
        _p(y_perm), _p(workspace), ws_bytes, _stream(stream)))


def moe_combine(shape, y_perm, slot_to_row, topk_weights, y, stream=None):
    _check("moe_combine", _lib.load().moe_combine(
        ctypes.byref(shape), _p(y_perm), _p(slot_to_row), _p(topk_weights), _p(y),
        _stream(stream)))


def moe_forward(shape, x, w_gate, router_bias, w1, w3, w2, w1_scale, w3_scale, w2_scale, y,
                topk_ids_out=None, topk_weights_out=None, expert_counts_out=None,
                drop_mask_out=None, logits_out=None, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("moe_forward", _lib.load().moe_forward(
        ctypes.byref(shape), _p(x), _p(w_gate), _p(router_bias), _p(w1), _p(w3), _p(w2),
        _p(w1_scale), _p(w3_scale), _p(w2_scale), _p(y), _p(topk_ids_out),
        _p(topk_weights_out), _p(expert_counts_out), _p(drop_mask_out), _p(logits_out),
        _p(workspace), ws_bytes, _stream(stream)))


def moe_forward_noalloc(shape, x, w_gate, router_bias, w1, w3, w2, w1_scale, w3_scale, w2_scale, y,
                        topk_ids_out=None, topk_weights_out=None, expert_counts_out=None,
                        drop_mask_out=None, logits_out=None, stream=None):
    _check("moe_forward_noalloc", _lib.load().moe_forward_noalloc(
        ctypes.byref(shape), _p(x), _p(w_gate), _p(router_bias), _p(w1), _p(w3), _p(w2),
        _p(w1_scale), _p(w3_scale), _p(w2_scale), _p(y), _p(topk_ids_out),
        _p(topk_weights_out), _p(expert_counts_out), _p(drop_mask_out), _p(logits_out),
        _stream(stream)))


# ---- scored routing, gradients of the gate, dense products ----

_TORCH = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def _ptr(fn: str, name: str, t, dtype, numel: int, dev: Optional[int]):
    """Address of one of a call's tensors, checked against the descriptor: element type, at least
    `numel` elements, contiguous, on device `dev` (a raw address passes unchecked)."""
    if t is None:
        return None
    try:
        if (t.get_device() == dev and (t.dtype is dtype or dtype is None) and t.numel() >= numel
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        return int(t)
    if not t.is_cuda:
        raise ValueError(f"{fn}: {name} must live in device memory")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{fn}: {name} needs {numel} elements, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous (row-major)")
    raise ValueError(f"{fn}: {name} is on device {t.get_device()}, another tensor on device {dev}")


def _device(*tensors) -> Optional[int]:
    """Index of the device of the first device tensor (None: raw addresses only)."""
    for t in tensors:
        if isinstance(t, torch.Tensor):
            d = t.get_device()
            if d >= 0:
                return d
    return None


def _workspace(fn: str, t, dev):
    """(address, bytes) of a workspace tensor or None."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{fn}: the workspace must be a tensor (its size is passed on)")
    return _ptr(fn, "workspace", t, None, 0, dev), t.numel() * t.element_size()


# The current stream's handle without building a Stream object (1.1 us less per call), and the
# current device without looking whether there is one (0.2 us less): a call with device tensors has.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(fn: str, dev: Optional[int], stream, *args):
    """The C call on `stream`, or on the current stream of the tensors' device; its launches go to that device."""
    f = getattr(_lib.load(), fn)
    if dev is None:
        _check(fn, f(*args, _stream(stream)))
    elif dev == _current_device():
        if stream is not None or _raw_stream is None:
            _check(fn, f(*args, _stream(stream)))
        else:
            _check(fn, f(*args, _raw_stream(dev)))
    else:
        with torch.cuda.device(dev):
            _check(fn, f(*args, _stream(stream)))


def make_router(score="softmax", n_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
                renormalize: bool = True, scale: float = 1.0) -> MoeRouter:
    return MoeRouter(_SCORE.get(score, score), n_groups, topk_groups, group_top, int(renormalize), scale)


def make_linear(M: int, N: int, K: int, dtype="bf16", y_dtype="bf16", act="none") -> MoeLinear:
    return MoeLinear(M, N, K, _DT.get(dtype, dtype), _DT.get(y_dtype, y_dtype), _ACT.get(act, act))


def moe_linear_workspace_bytes(linear: MoeLinear, call: int = MOE_CALL_LINEAR) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_linear_workspace_bytes", _lib.load().moe_linear_workspace_bytes(
        ctypes.byref(linear), call, ctypes.byref(n)))
    return n.value


def moe_linear(linear, x, w, bias, residual, y, pre=None, workspace=None, stream=None):
    fn = "moe_linear"
    M, N, K = linear.M, linear.N, linear.K
    dt, ydt, d = _TORCH.get(linear.dtype), _TORCH.get(linear.y_dtype), _device(x, w, y)
    _run(fn, d, stream, ctypes.byref(linear), _ptr(fn, "x", x, dt, M * K, d), _ptr(fn, "w", w, dt, N * K, d),
         _ptr(fn, "bias", bias, torch.float32, N, d), _ptr(fn, "residual", residual, ydt, M * N, d),
         _ptr(fn, "y", y, ydt, M * N, d), _ptr(fn, "pre", pre, dt, M * N, d), *_workspace(fn, workspace, d))


def moe_linear_backward(linear, dy, pre, x, w, dx, dw, dbias, workspace=None, stream=None):
    fn = "moe_linear_backward"
    M, N, K = linear.M, linear.N, linear.K
    dt, ydt, d = _TORCH.get(linear.dtype), _TORCH.get(linear.y_dtype), _device(dy, x, w, dx, dw, dbias)
    _run(fn, d, stream, ctypes.byref(linear), _ptr(fn, "dy", dy, ydt, M * N, d),
         _ptr(fn, "pre", pre, dt, M * N, d), _ptr(fn, "x", x, dt, M * K, d), _ptr(fn, "w", w, dt, N * K, d),
         _ptr(fn, "dx", dx, dt, M * K, d), _ptr(fn, "dw", dw, dt, N * K, d),
         _ptr(fn, "dbias", dbias, torch.float32, N, d), *_workspace(fn, workspace, d))


def moe_route_scored(shape, router, logits, balance_bias, topk_ids, topk_weights, scores=None,
                     next_ids=None, stream=None):
    fn = "moe_route_scored"
    T, E, k = shape.T, shape.n_experts, shape.top_k
    f32, i32, d = torch.float32, torch.int32, _device(logits, topk_ids, topk_weights)
    _run(fn, d, stream, ctypes.byref(shape), ctypes.byref(router), _ptr(fn, "logits", logits, f32, T * E, d),
         _ptr(fn, "balance_bias", balance_bias, f32, E, d), _ptr(fn, "topk_ids", topk_ids, i32, T * k, d),
         _ptr(fn, "topk_weights", topk_weights, f32, T * k, d), _ptr(fn, "scores", scores, f32, T * E, d),
         _ptr(fn, "next_ids", next_ids, i32, T * 2, d))


def moe_route_scored_backward(shape, router, logits, topk_ids, dweights, dscores, dlogits, stream=None):
    fn = "moe_route_scored_backward"
    T, E, k = shape.T, shape.n_experts, shape.top_k
    f32, d = torch.float32, _device(logits, dweights, dlogits)
    _run(fn, d, stream, ctypes.byref(shape), ctypes.byref(router), _ptr(fn, "logits", logits, f32, T * E, d),
         _ptr(fn, "topk_ids", topk_ids, torch.int32, T * k, d), _ptr(fn, "dweights", dweights, f32, T * k, d),
         _ptr(fn, "dscores", dscores, f32, T * E, d), _ptr(fn, "dlogits", dlogits, f32, T * E, d))


def moe_combine_backward(shape, dy, y_perm, slot_to_row, topk_weights, dy_perm, dweights, stream=None):
    fn = "moe_combine_backward"
    T, dm, k = shape.T, shape.d_model, shape.top_k
    R = T * (k + shape.n_shared)
    f32, dt, d = torch.float32, _TORCH.get(shape.act_dtype), _device(dy, slot_to_row, topk_weights)
    _run(fn, d, stream, ctypes.byref(shape), _ptr(fn, "dy", dy, dt, T * dm, d),
         _ptr(fn, "y_perm", y_perm, f32, R * dm, d), _ptr(fn, "slot_to_row", slot_to_row, torch.int32, R, d),
         _ptr(fn, "topk_weights", topk_weights, f32, T * k, d), _ptr(fn, "dy_perm", dy_perm, dt, R * dm, d),
         _ptr(fn, "dweights", dweights, f32, T * k, d))


def moe_forward_routed(shape, x, topk_ids, topk_weights, next_ids, w1, w3, w2, w1_scale, w3_scale,
                       w2_scale, y, expert_counts_out=None, drop_mask_out=None, workspace=None,
                       stream=None):
    fn = "moe_forward_routed"
    T, dm, dff, k, G = shape.T, shape.d_model, shape.d_ff, shape.top_k, shape.n_experts + shape.n_shared
    dt, i32, d = _TORCH.get(shape.act_dtype), torch.int32, _device(x, topk_ids, topk_weights, y)
    # expert weights and scales in their storage types
    wt, n_w, st, n_up, n_down = _TORCH.get(shape.w_dtype), G * dm * dff, None, 0, 0
    if shape.w_dtype == MOE_FP8_E4M3:
        st, n_up, n_down = torch.float32, G * dff, G * dm
    elif shape.w_dtype == MOE_MXFP4:
        n_w, st, n_up, n_down = n_w // 2, torch.uint8, n_w // 32, n_w // 32
    _run(fn, d, stream, ctypes.byref(shape), _ptr(fn, "x", x, dt, T * dm, d),
         _ptr(fn, "topk_ids", topk_ids, i32, T * k, d),
         _ptr(fn, "topk_weights", topk_weights, torch.float32, T * k, d),
         _ptr(fn, "next_ids", next_ids, i32, T * 2, d), _ptr(fn, "w1", w1, wt, n_w, d),
         _ptr(fn, "w3", w3, wt, n_w, d), _ptr(fn, "w2", w2, wt, n_w, d),
         _ptr(fn, "w1_scale", w1_scale, st, n_up, d), _ptr(fn, "w3_scale", w3_scale, st, n_up, d),
         _ptr(fn, "w2_scale", w2_scale, st, n_down, d), _ptr(fn, "y", y, dt, T * dm, d),
         _ptr(fn, "expert_counts_out", expert_counts_out, i32, G, d),
         _ptr(fn, "drop_mask_out", drop_mask_out, torch.uint8, T * k, d), *_workspace(fn, workspace, d))
