"""Python binding of librdot, the GB300 (sm_103a) ragged-dot / Group-GEMM library.

Argument marshalling only: every step of the computation runs in the library's CUDA kernels.
PyTorch supplies device memory and streams. The low-level functions carry the C ABI's names
(``rdot_plan``, ``rdot_forward``, ...) and take torch tensors; :class:`Plan` and
:func:`ragged_dot` are conveniences over them.

There is no fallback: if ``librdot.so`` has not been built (``group_gemm_gb300.build()``), or
the device is not an sm_10x GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import _build

__all__ = [
    "build", "load", "RdotError", "Problem", "Plan",
    "rdot_plan", "rdot_plan_destroy", "rdot_workspace_size", "rdot_forward", "rdot_forward_mxfp8",
    "rdot_grad_weight", "rdot_padded_workspace_size", "rdot_padded_forward", "rdot_read_status",
    "rdot_clear_status", "rdot_debug_offsets_tilemap", "rdot_plan_info", "rdot_debug_wait_timeout",
    "rdot_set_wait_timeout", "rdot_status_string", "rdot_last_cuda_error", "rdot_version",
    "rdot_forward_no_alloc", "rdot_no_alloc_read_status", "rdot_grad_input", "rdot_moe_route_workspace_size",
    "rdot_moe_permute", "rdot_moe_unpermute", "rdot_forward_gated", "rdot_grad_input_mxfp8", "rdot_router_topk",
    "rdot_forward_combine", "rdot_grad_weight_mxfp8", "router_topk", "ragged_dot_combine", "grad_weight_mxfp8",
    "moe_permute", "moe_unpermute", "ragged_dot", "grad_weight",
    "grad_input", "ragged_dot_gated",
    "ragged_dot_mxfp8", "padded_ragged_dot",
    "rdot_moe_unpermute_grad", "rdot_moe_permute_grad", "rdot_router_topk_grad",
    "rdot_quantize_mxfp4", "rdot_quantize_mxfp4_weight", "rdot_mxfp4_weight_scale_bytes", "rdot_forward_mxfp4",
    "quantize_mxfp4", "quantize_mxfp4_weight", "ragged_dot_mxfp4",
    "moe_unpermute_grad", "moe_permute_grad", "router_topk_grad", "EXPORTED_SYMBOLS",
]

RDOT_OK, RDOT_ERR_INVALID_ARG, RDOT_ERR_UNSUPPORTED, RDOT_ERR_CUDA = 0, 1, 2, 3
RDOT_ERR_DEVICE_TIMEOUT, RDOT_WARN_GROUP_SIZES = 4, 5
RDOT_F32, RDOT_BF16, RDOT_E4M3, RDOT_E2M1 = 0, 1, 2, 3
RDOT_MODE_FORWARD, RDOT_MODE_GRAD_WEIGHT, RDOT_MODE_FORWARD_MXFP8, RDOT_MODE_GRAD_INPUT = 0, 1, 2, 3
RDOT_MODE_FORWARD_GATED, RDOT_MODE_GRAD_INPUT_MXFP8, RDOT_MODE_GRAD_WEIGHT_MXFP8 = 4, 5, 6
RDOT_MODE_FORWARD_MXFP4 = 8
RDOT_STATUS_BIT_GROUP_SIZES, RDOT_STATUS_BIT_TIMEOUT = 0x1, 0x2
RDOT_FLAG_ROW_TILES_INNER, RDOT_FLAG_COL_TILES_INNER = 0x1, 0x2
RDOT_FLAG_CTA_PAIR, RDOT_FLAG_NO_CTA_PAIR, RDOT_FLAG_NATURAL_ORDER = 0x4, 0x8, 0x10
RDOT_FLAG_SKINNY, RDOT_FLAG_NO_SKINNY = 0x20, 0x40
RDOT_MAX_GROUPS = 1024
RDOT_ROUTER_VALUES, RDOT_ROUTER_SOFTMAX, RDOT_ROUTER_SOFTMAX_TOPK, RDOT_ROUTER_MAX_TOPK = 0, 1, 2, 32
_ROUTER_MODES = {"values": RDOT_ROUTER_VALUES, "softmax": RDOT_ROUTER_SOFTMAX, "softmax_topk": RDOT_ROUTER_SOFTMAX_TOPK}

# every function include/rdot.h declares
EXPORTED_SYMBOLS = (
    "rdot_plan", "rdot_plan_destroy", "rdot_workspace_size", "rdot_forward", "rdot_forward_mxfp8",
    "rdot_grad_weight", "rdot_padded_workspace_size", "rdot_padded_forward", "rdot_read_status",
    "rdot_clear_status", "rdot_debug_offsets_tilemap", "rdot_plan_info", "rdot_debug_wait_timeout",
    "rdot_set_wait_timeout", "rdot_status_string", "rdot_last_cuda_error", "rdot_version",
    "rdot_forward_no_alloc", "rdot_no_alloc_read_status", "rdot_grad_input", "rdot_moe_route_workspace_size",
    "rdot_moe_permute", "rdot_moe_unpermute", "rdot_forward_gated", "rdot_grad_input_mxfp8", "rdot_router_topk",
    "rdot_forward_combine", "rdot_grad_weight_mxfp8",
    "rdot_moe_unpermute_grad", "rdot_moe_permute_grad", "rdot_router_topk_grad",
    "rdot_quantize_mxfp4", "rdot_quantize_mxfp4_weight", "rdot_mxfp4_weight_scale_bytes", "rdot_forward_mxfp4",
)

_DTYPE_CODES = {"f32": RDOT_F32, "bf16": RDOT_BF16, "e4m3": RDOT_E4M3, "e2m1": RDOT_E2M1}
_MODE_CODES = {"forward": RDOT_MODE_FORWARD, "grad_weight": RDOT_MODE_GRAD_WEIGHT,
               "forward_mxfp8": RDOT_MODE_FORWARD_MXFP8, "grad_input": RDOT_MODE_GRAD_INPUT,
               "forward_gated": RDOT_MODE_FORWARD_GATED, "grad_input_mxfp8": RDOT_MODE_GRAD_INPUT_MXFP8,
               "grad_weight_mxfp8": RDOT_MODE_GRAD_WEIGHT_MXFP8, "forward_mxfp4": RDOT_MODE_FORWARD_MXFP4}


class RdotError(RuntimeError):
    def __init__(self, status: int, what: str):
        lib = _lib
        name = lib.rdot_status_string(status).decode() if lib else str(status)
        detail = lib.rdot_last_cuda_error().decode() if (lib and status == RDOT_ERR_CUDA) else ""
        super().__init__(f"{what}: {name}" + (f" ({detail})" if detail else ""))
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("k", ctypes.c_int64), ("n", ctypes.c_int64),
                ("groups", ctypes.c_int32), ("mode", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("flags", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile librdot.so in-tree for sm_103a."""
    return _build.build(force=force, verbose=verbose)


def load():
    """Loads librdot.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"librdot.so is not built ({_build.LIB}); call group_gemm_gb300.build()")
        lib = ctypes.CDLL(_build.LIB)
        vp, st = ctypes.c_void_p, ctypes.c_int
        i32p, i64 = ctypes.POINTER(ctypes.c_int32), ctypes.c_int64
        sig = {
            "rdot_plan": ([ctypes.POINTER(Problem), ctypes.c_int, ctypes.POINTER(vp)], st),
            "rdot_plan_destroy": ([vp], st),
            "rdot_workspace_size": ([vp, ctypes.POINTER(ctypes.c_size_t)], st),
            "rdot_forward": ([vp, vp, vp, vp, vp, vp, vp], st),
            "rdot_forward_mxfp8": ([vp, vp, vp, vp, vp, vp, vp, vp, vp], st),
            "rdot_grad_weight": ([vp, vp, vp, vp, vp, vp, vp], st),
            "rdot_grad_input": ([vp, vp, vp, vp, vp, vp, vp], st),
            "rdot_forward_gated": ([vp, vp, vp, vp, vp, vp, vp, vp], st),
            "rdot_grad_input_mxfp8": ([vp, vp, vp, vp, vp, vp, vp, vp, vp], st),
            "rdot_moe_route_workspace_size": ([i64, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
                                              st),
            "rdot_moe_permute": ([vp, i64, ctypes.c_int32, ctypes.c_int32, vp, i64, vp, vp, vp, vp, vp, vp], st),
            "rdot_moe_unpermute": ([vp, vp, vp, i64, ctypes.c_int32, i64, vp, vp], st),
            "rdot_padded_workspace_size": ([vp, i64, ctypes.POINTER(ctypes.c_size_t)], st),
            "rdot_padded_forward": ([vp, vp, vp, vp, vp, i64, vp, vp, vp], st),
            "rdot_read_status": ([vp, vp, i32p, vp], st),
            "rdot_clear_status": ([vp, vp, vp], st),
            "rdot_debug_offsets_tilemap": ([vp, vp, vp, vp, vp, i64, vp, vp], st),
            "rdot_plan_info": ([vp, i32p, i32p, i32p, i32p], st),
            "rdot_debug_wait_timeout": ([vp, ctypes.c_uint64, vp, vp], st),
            "rdot_set_wait_timeout": ([vp, ctypes.c_uint64], st),
            "rdot_status_string": ([st], ctypes.c_char_p),
            "rdot_last_cuda_error": ([], ctypes.c_char_p),
            "rdot_version": ([], ctypes.c_int),
            "rdot_forward_no_alloc": ([vp, vp, vp, vp, vp, vp], st),
            "rdot_no_alloc_read_status": ([vp, i32p, vp], st),
            "rdot_grad_weight_mxfp8": ([vp, vp, vp, vp, vp, vp, vp, vp, vp], st),
            "rdot_forward_combine": ([vp, vp, vp, vp, vp, vp, i64, ctypes.c_int32, vp, vp, vp], st),
            "rdot_router_topk": ([vp, ctypes.c_int32, i64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp, vp],
                                 st),
            "rdot_quantize_mxfp4": ([vp, ctypes.c_int32, i64, i64, vp, vp, vp, vp], st),
            "rdot_quantize_mxfp4_weight": ([vp, ctypes.c_int32, ctypes.c_int32, i64, i64, vp, vp, vp, vp], st),
            "rdot_mxfp4_weight_scale_bytes": ([ctypes.c_int32, i64, i64, ctypes.POINTER(ctypes.c_size_t)], st),
            "rdot_forward_mxfp4": ([vp, vp, vp, vp, vp, vp, vp, vp, vp], st),
            "rdot_moe_unpermute_grad": ([vp, vp, vp, vp, vp, i64, ctypes.c_int32, i64, vp, vp, vp], st),
            "rdot_moe_permute_grad": ([vp, ctypes.c_int32, vp, i64, ctypes.c_int32, i64, vp, vp], st),
            "rdot_router_topk_grad": ([vp, ctypes.c_int32, vp, vp, vp, i64, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_int32, vp, vp], st),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
        return lib


def _check(status: int, what: str):
    if status != RDOT_OK:
        raise RdotError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    """The cudaStream_t of a torch stream, a raw handle, or (None) the device's current stream. The last
    is asked for as a raw handle where a tensor's device is given: building a torch.cuda.Stream costs more than
    the library's own call. Any other device (None: the current one) is torch.cuda.current_stream's to resolve."""
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and isinstance(device, torch.device) and device.type == "cuda" and device.index is not None:
            return raw(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ------------------------------------------------------------------------------ C-ABI names
def rdot_plan(problem: Problem, device: int = 0) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load().rdot_plan(ctypes.byref(problem), int(device), ctypes.byref(h)), "rdot_plan")
    return h


def rdot_plan_destroy(plan) -> None:
    _check(load().rdot_plan_destroy(plan), "rdot_plan_destroy")


def rdot_workspace_size(plan) -> int:
    n = ctypes.c_size_t()
    _check(load().rdot_workspace_size(plan, ctypes.byref(n)), "rdot_workspace_size")
    return n.value


def rdot_forward(plan, lhs, rhs, group_sizes, out, workspace, stream=None) -> None:
    _check(load().rdot_forward(plan, _ptr(lhs), _ptr(rhs), _ptr(group_sizes), _ptr(out), _ptr(workspace),
                               _stream(stream, out.device)), "rdot_forward")


def rdot_forward_mxfp8(plan, lhs, lhs_scale, rhs, rhs_scale, group_sizes, out, workspace, stream=None) -> None:
    _check(load().rdot_forward_mxfp8(plan, _ptr(lhs), _ptr(lhs_scale), _ptr(rhs), _ptr(rhs_scale),
                                     _ptr(group_sizes), _ptr(out), _ptr(workspace),
                                     _stream(stream, out.device)), "rdot_forward_mxfp8")


def rdot_grad_weight(plan, lhs, dy, group_sizes, dw, workspace, stream=None) -> None:
    _check(load().rdot_grad_weight(plan, _ptr(lhs), _ptr(dy), _ptr(group_sizes), _ptr(dw), _ptr(workspace),
                                   _stream(stream, dw.device)), "rdot_grad_weight")


def rdot_grad_input(plan, dy, rhs, group_sizes, dlhs, workspace, stream=None) -> None:
    _check(load().rdot_grad_input(plan, _ptr(dy), _ptr(rhs), _ptr(group_sizes), _ptr(dlhs), _ptr(workspace),
                                  _stream(stream, dlhs.device)), "rdot_grad_input")


def rdot_grad_input_mxfp8(plan, dy_q, dy_scale, w_q, w_scale, group_sizes, dlhs, workspace, stream=None) -> None:
    _check(load().rdot_grad_input_mxfp8(plan, _ptr(dy_q), _ptr(dy_scale), _ptr(w_q), _ptr(w_scale),
                                        _ptr(group_sizes), _ptr(dlhs), _ptr(workspace),
                                        _stream(stream, dlhs.device)), "rdot_grad_input_mxfp8")


def rdot_forward_gated(plan, lhs, w0, w1, group_sizes, out, workspace, stream=None) -> None:
    _check(load().rdot_forward_gated(plan, _ptr(lhs), _ptr(w0), _ptr(w1), _ptr(group_sizes), _ptr(out),
                                     _ptr(workspace), _stream(stream, out.device)), "rdot_forward_gated")


def rdot_moe_route_workspace_size(tokens: int, topk: int, n_experts: int) -> int:
    n = ctypes.c_size_t()
    _check(load().rdot_moe_route_workspace_size(int(tokens), int(topk), int(n_experts), ctypes.byref(n)),
           "rdot_moe_route_workspace_size")
    return n.value


def rdot_moe_permute(topk_ids, x, n_experts, group_sizes, order, inv, x_sorted, workspace, stream=None) -> None:
    t, k = topk_ids.shape
    _check(load().rdot_moe_permute(_ptr(topk_ids), int(t), int(k), int(n_experts), _ptr(x),
                                   int(x.shape[1] * x.element_size()), _ptr(group_sizes), _ptr(order), _ptr(inv),
                                   _ptr(x_sorted), _ptr(workspace), _stream(stream, x.device)), "rdot_moe_permute")


def rdot_moe_unpermute(y_sorted, inv, topk_weights, out, stream=None) -> None:
    t, k = topk_weights.shape
    _check(load().rdot_moe_unpermute(_ptr(y_sorted), _ptr(inv), _ptr(topk_weights), int(t), int(k),
                                     int(y_sorted.shape[1]), _ptr(out), _stream(stream, out.device)),
           "rdot_moe_unpermute")


def rdot_grad_weight_mxfp8(plan, lhs_q, lhs_s, dy_q, dy_s, group_sizes, dw, workspace, stream=None) -> None:
    _check(load().rdot_grad_weight_mxfp8(plan, _ptr(lhs_q), _ptr(lhs_s), _ptr(dy_q), _ptr(dy_s), _ptr(group_sizes),
                                         _ptr(dw), _ptr(workspace), _stream(stream, dw.device)),
           "rdot_grad_weight_mxfp8")


def rdot_forward_combine(plan, lhs, rhs, group_sizes, order, topk_weights, out, workspace, stream=None) -> None:
    """Down projection with the router-weighted un-permute fused: out fp32 [T, N]."""
    t, k = topk_weights.shape
    _check(load().rdot_forward_combine(plan, _ptr(lhs), _ptr(rhs), _ptr(group_sizes), _ptr(order),
                                       _ptr(topk_weights), int(t), int(k), _ptr(out), _ptr(workspace),
                                       _stream(stream, out.device)), "rdot_forward_combine")


def rdot_router_topk(logits, topk: int, weights_mode: int, topk_ids, topk_weights, stream=None) -> None:
    """logits [T, E] fp32 or bf16 -> topk_ids int32 [T, k], topk_weights fp32 [T, k]."""
    import torch
    t, e = logits.shape
    dt = {torch.float32: RDOT_F32, torch.bfloat16: RDOT_BF16}.get(logits.dtype)
    if dt is None:
        raise TypeError("logits must be float32 or bfloat16")
    _check(load().rdot_router_topk(_ptr(logits), dt, int(t), int(e), int(topk), int(weights_mode), _ptr(topk_ids),
                                   _ptr(topk_weights), _stream(stream, logits.device)), "rdot_router_topk")


def _float_dtype(t, what: str) -> int:
    import torch
    dt = {torch.float32: RDOT_F32, torch.bfloat16: RDOT_BF16}.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what} must be float32 or bfloat16")
    return dt


def rdot_quantize_mxfp4(x, codes, scales, values=None, stream=None) -> None:
    """x [rows, K] (fp32 or bf16) -> codes uint8 [rows, K/2], scales uint8 [rows, K/32], values bf16 [rows, K]."""
    _check(load().rdot_quantize_mxfp4(_ptr(x), _float_dtype(x, "x"), int(x.shape[0]), int(x.shape[1]), _ptr(codes),
                                      _ptr(scales), _ptr(values), _stream(stream, x.device)), "rdot_quantize_mxfp4")


def rdot_mxfp4_weight_scale_bytes(groups: int, k: int, n: int) -> int:
    b = ctypes.c_size_t()
    _check(load().rdot_mxfp4_weight_scale_bytes(int(groups), int(k), int(n), ctypes.byref(b)),
           "rdot_mxfp4_weight_scale_bytes")
    return b.value


def rdot_quantize_mxfp4_weight(w, codes, scales, values=None, stream=None) -> None:
    """w [G, K, N] (fp32 or bf16) -> codes uint8 [G, N, K/2], scales uint8 [G, ceil(N/128), ceil(K/128), 512],
    values bf16 [G, K, N]."""
    g, k, n = w.shape
    _check(load().rdot_quantize_mxfp4_weight(_ptr(w), _float_dtype(w, "w"), int(g), int(k), int(n), _ptr(codes),
                                             _ptr(scales), _ptr(values), _stream(stream, w.device)),
           "rdot_quantize_mxfp4_weight")


def rdot_forward_mxfp4(plan, lhs, lhs_scale, rhs, rhs_scale, group_sizes, out, workspace, stream=None) -> None:
    _check(load().rdot_forward_mxfp4(plan, _ptr(lhs), _ptr(lhs_scale), _ptr(rhs), _ptr(rhs_scale),
                                     _ptr(group_sizes), _ptr(out), _ptr(workspace), _stream(stream, out.device)),
           "rdot_forward_mxfp4")


def rdot_moe_unpermute_grad(dout, y_sorted, order, inv, topk_weights, dy_sorted, dweights, stream=None) -> None:
    """dout bf16 [T, N], y_sorted bf16 [T*k, N] -> dy_sorted bf16 [T*k, N], dweights fp32 [T, k]."""
    t, k = topk_weights.shape
    _check(load().rdot_moe_unpermute_grad(_ptr(dout), _ptr(y_sorted), _ptr(order), _ptr(inv), _ptr(topk_weights),
                                          int(t), int(k), int(y_sorted.shape[1]), _ptr(dy_sorted), _ptr(dweights),
                                          _stream(stream, dout.device)), "rdot_moe_unpermute_grad")


def rdot_moe_permute_grad(dx_sorted, inv, dx, stream=None) -> None:
    """dx_sorted [T*k, N] (fp32 or bf16) -> dx [T, N], the same dtype."""
    if dx.dtype != dx_sorted.dtype:
        raise TypeError("dx must have dx_sorted's dtype")
    t = dx.shape[0]
    _check(load().rdot_moe_permute_grad(_ptr(dx_sorted), _float_dtype(dx_sorted, "dx_sorted"), _ptr(inv), int(t),
                                        inv.numel() // t if t else 1, int(dx.shape[1]), _ptr(dx),
                                        _stream(stream, dx.device)), "rdot_moe_permute_grad")


def rdot_router_topk_grad(logits, topk_ids, topk_weights, dweights, weights_mode: int, dlogits, stream=None) -> None:
    """The logits' gradient, dlogits [T, E] (fp32 or bf16), from the weights' (fp32 [T, k]); logits
    (the same dtype) may be None unless the weights are the softmax over all experts."""
    if logits is not None and logits.dtype != dlogits.dtype:
        raise TypeError("logits must have dlogits' dtype")
    t, e = dlogits.shape
    _check(load().rdot_router_topk_grad(_ptr(logits), _float_dtype(dlogits, "dlogits"), _ptr(topk_ids),
                                        _ptr(topk_weights), _ptr(dweights), int(t), int(e), int(topk_ids.shape[1]),
                                        int(weights_mode), _ptr(dlogits), _stream(stream, dlogits.device)),
           "rdot_router_topk_grad")


def rdot_padded_workspace_size(plan, capacity: int) -> int:
    n = ctypes.c_size_t()
    _check(load().rdot_padded_workspace_size(plan, int(capacity), ctypes.byref(n)), "rdot_padded_workspace_size")
    return n.value


def rdot_padded_forward(plan, lhs, rhs, group_sizes, out, capacity, pad_workspace, workspace, stream=None):
    _check(load().rdot_padded_forward(plan, _ptr(lhs), _ptr(rhs), _ptr(group_sizes), _ptr(out), int(capacity),
                                      _ptr(pad_workspace), _ptr(workspace), _stream(stream, out.device)),
           "rdot_padded_forward")


def rdot_read_status(plan, workspace, stream=None) -> int:
    """Returns the status bit word (synchronises the stream)."""
    v = ctypes.c_int32()
    st = load().rdot_read_status(plan, _ptr(workspace), ctypes.byref(v), _stream(stream, workspace.device))
    if st not in (RDOT_OK, RDOT_ERR_DEVICE_TIMEOUT, RDOT_WARN_GROUP_SIZES):
        _check(st, "rdot_read_status")
    return v.value


def rdot_clear_status(plan, workspace, stream=None) -> None:
    _check(load().rdot_clear_status(plan, _ptr(workspace), _stream(stream, workspace.device)), "rdot_clear_status")


def rdot_debug_offsets_tilemap(plan, group_sizes, offsets, tile_prefix, tiles=None, workspace=None,
                               stream=None) -> None:
    max_tiles = 0 if tiles is None else tiles.shape[0]
    _check(load().rdot_debug_offsets_tilemap(plan, _ptr(group_sizes), _ptr(offsets), _ptr(tile_prefix),
                                             _ptr(tiles), int(max_tiles), _ptr(workspace),
                                             _stream(stream, group_sizes.device)), "rdot_debug_offsets_tilemap")


def rdot_plan_info(plan):
    vals = [ctypes.c_int32() for _ in range(4)]
    _check(load().rdot_plan_info(plan, *[ctypes.byref(v) for v in vals]), "rdot_plan_info")
    return dict(zip(("tile_m", "tile_n", "m_inner", "grid_ctas"), (v.value for v in vals)))


def rdot_debug_wait_timeout(plan, timeout_ns: int, workspace, stream=None) -> None:
    _check(load().rdot_debug_wait_timeout(plan, int(timeout_ns), _ptr(workspace),
                                          _stream(stream, workspace.device)), "rdot_debug_wait_timeout")


def rdot_set_wait_timeout(plan, timeout_ns: int) -> None:
    _check(load().rdot_set_wait_timeout(plan, int(timeout_ns)), "rdot_set_wait_timeout")


def rdot_forward_no_alloc(plan, lhs, rhs, group_sizes, out, stream=None) -> None:
    """Forward with the library's static device scratch instead of a caller workspace."""
    _check(load().rdot_forward_no_alloc(plan, _ptr(lhs), _ptr(rhs), _ptr(group_sizes), _ptr(out),
                                        _stream(stream, out.device)), "rdot_forward_no_alloc")


def rdot_no_alloc_read_status(plan, stream=None, device=None):
    """Returns ``(status, flags)``: the status word the last rdot_forward_no_alloc call on the
    plan's device left in the library's static scratch (synchronises the stream)."""
    v = ctypes.c_int32()
    st = load().rdot_no_alloc_read_status(plan, ctypes.byref(v), _stream(stream, device))
    if st not in (RDOT_OK, RDOT_WARN_GROUP_SIZES, RDOT_ERR_DEVICE_TIMEOUT):
        raise RdotError(st, "rdot_no_alloc_read_status")
    return st, v.value


def rdot_status_string(status: int) -> str:
    return load().rdot_status_string(int(status)).decode()


def rdot_last_cuda_error() -> str:
    return load().rdot_last_cuda_error().decode()


def rdot_version() -> int:
    return load().rdot_version()


# ------------------------------------------------------------------------------ conveniences
class Plan:
    """Owns an ``rdot_plan_t`` and a zeroed workspace on ``device``."""

    def __init__(self, m, k, n, groups, mode="forward", in_dtype="bf16", out_dtype="bf16", device=0,
                 tile_n=0, flags=0):
        import torch
        self.problem = Problem(m=int(m), k=int(k), n=int(n), groups=int(groups), mode=_MODE_CODES[mode],
                               in_dtype=_DTYPE_CODES[in_dtype], out_dtype=_DTYPE_CODES[out_dtype],
                               tile_n=int(tile_n), flags=int(flags))
        self.device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
        self.handle = rdot_plan(self.problem, self.device.index or 0)
        self.workspace = torch.zeros(rdot_workspace_size(self.handle) // 4, dtype=torch.int32, device=self.device)
        self._workspaces = {torch.cuda.current_stream(self.device).cuda_stream: self.workspace}
        self.info = rdot_plan_info(self.handle)

    def workspace_on(self, stream):
        """A zeroed workspace for calls on ``stream`` (a torch stream), allocated on that stream
        the first time: calls rewrite their workspace (status word, MXFP8 scale blocks,
        grad-weight maps), so calls that may run concurrently on different streams get their own."""
        import torch
        ws = self._workspaces.get(stream.cuda_stream)
        if ws is None:
            with torch.cuda.stream(stream):
                ws = torch.zeros_like(self.workspace)
            self._workspaces[stream.cuda_stream] = ws
        return ws

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.rdot_plan_destroy(h)
            self.handle = None

    def status(self, stream=None) -> int:
        return rdot_read_status(self.handle, self.workspace, stream)

    def clear_status(self, stream=None) -> None:
        rdot_clear_status(self.handle, self.workspace, stream)


_plan_cache = {}


def _run_stream(stream, device):
    """The torch stream a high-level call runs on: ``stream`` (a torch stream, or a raw
    cudaStream_t as an int, 0 meaning the legacy default stream) or the device's current stream."""
    import torch
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if int(stream) == 0:
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(int(stream), device=device)


def _cached_plan(key, stream, **kw):
    """The plan for a shape (host state, shared by all streams) and its workspace on ``stream``."""
    p = _plan_cache.get(key)
    if p is None:
        p = Plan(**kw)
        _plan_cache[key] = p
    return p, p.workspace_on(stream)


def _torch_dtype_name(dt):
    import torch
    return {torch.float32: "f32", torch.bfloat16: "bf16"}[dt]


def _check_out(out, elements, dtype, device, what="out"):
    """Refuses a caller's output that a kernel, which gets its pointer alone, would write past the end of or
    with values of another type or order."""
    if out.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}")
    if out.numel() < elements or not out.is_contiguous() or out.device != device:
        raise ValueError(f"{what} must be contiguous, of at least {elements} elements, on {device}")


def _same_device(*tensors):
    """Refuses tensors of several devices: a kernel would follow a pointer that is not its device's."""
    if any(t.device != tensors[0].device for t in tensors):
        raise ValueError("all tensors must be on one device")


# The high-level calls below allocate what they return (and any scratch) on the stream their
# kernels run on, so PyTorch's caching allocator never hands that memory to other work while
# those kernels may still use it.

def ragged_dot(lhs, rhs, group_sizes, out_dtype=None, out=None, stream=None):
    """``out[i, :] = lhs[i, :] @ rhs[g(i)]`` with rows past ``sum(group_sizes)`` zero.

    lhs [M, K] and rhs [G, K, N] (both fp32 or both bf16) and group_sizes int32 [G] live on the
    same CUDA device. Returns out [M, N] (``out_dtype`` defaults to the input dtype)."""
    import torch
    m, k = lhs.shape
    g, k2, n = rhs.shape
    if k2 != k or group_sizes.shape != (g,):
        raise ValueError("shape mismatch between lhs, rhs and group_sizes")
    in_dt = _torch_dtype_name(lhs.dtype)
    out_dtype = out_dtype or lhs.dtype
    if out is not None:
        _check_out(out, m * n, out_dtype, lhs.device)
    s = _run_stream(stream, lhs.device)
    key = ("fwd", m, k, n, g, in_dt, out_dtype, lhs.device)
    plan, ws = _cached_plan(key, s, m=m, k=k, n=n, groups=g, mode="forward", in_dtype=in_dt,
                            out_dtype=_torch_dtype_name(out_dtype), device=lhs.device)
    with torch.cuda.stream(s):
        if out is None:
            out = torch.empty((m, n), dtype=out_dtype, device=lhs.device)
        rdot_forward(plan.handle, lhs.contiguous(), rhs.contiguous(), group_sizes.to(torch.int32).contiguous(), out,
                     ws, s)
    return out


def grad_weight(lhs, dy, group_sizes, out_dtype=None, dw=None, stream=None):
    """``dw[g] = lhs_g^T dy_g`` ([G, K, N], fp32 by default or bf16) for bf16 lhs [M, K] and
    dy [M, N]."""
    import torch
    m, k = lhs.shape
    _, n = dy.shape
    g = group_sizes.shape[0]
    out_dtype = out_dtype or (dw.dtype if dw is not None else torch.float32)
    if dw is not None:
        _check_out(dw, g * k * n, out_dtype, lhs.device, "dw")
    names = {torch.bfloat16: "bf16", torch.float32: "f32"}
    s = _run_stream(stream, lhs.device)
    key = ("wgrad", m, k, n, g, out_dtype, lhs.device)
    plan, ws = _cached_plan(key, s, m=m, k=k, n=n, groups=g, mode="grad_weight", in_dtype="bf16",
                            out_dtype=names[out_dtype], device=lhs.device)
    with torch.cuda.stream(s):
        if dw is None:
            dw = torch.empty((g, k, n), dtype=out_dtype, device=lhs.device)
        rdot_grad_weight(plan.handle, lhs.contiguous(), dy.contiguous(), group_sizes.to(torch.int32).contiguous(),
                         dw, ws, s)
    return dw


def grad_input(dy, rhs, group_sizes, out_dtype=None, dlhs=None, stream=None):
    """``dlhs[i] = dy[i] @ rhs[g(i)]^T`` ([M, K]) for bf16 dy [M, N] and rhs [G, K, N]: the
    data gradient of :func:`ragged_dot` (zeros past the sum)."""
    import torch
    m, n = dy.shape
    g, k, _ = rhs.shape
    out_dtype = out_dtype or dy.dtype
    if dlhs is not None:
        _check_out(dlhs, m * k, out_dtype, dy.device, "dlhs")
    names = {torch.bfloat16: "bf16", torch.float32: "f32"}
    s = _run_stream(stream, dy.device)
    key = ("dgrad", m, k, n, g, out_dtype, dy.device)
    plan, ws = _cached_plan(key, s, m=m, k=k, n=n, groups=g, mode="grad_input", in_dtype="bf16",
                            out_dtype=names[out_dtype], device=dy.device)
    with torch.cuda.stream(s):
        if dlhs is None:
            dlhs = torch.empty((m, k), dtype=out_dtype, device=dy.device)
        rdot_grad_input(plan.handle, dy.contiguous(), rhs.contiguous(), group_sizes.to(torch.int32).contiguous(),
                        dlhs, ws, s)
    return dlhs


def ragged_dot_gated(lhs, w0, w1, group_sizes, out_dtype=None, out=None, stream=None):
    """``silu(lhs @ w0[g]) * (lhs @ w1[g])`` for bf16 lhs [M, K], w0/w1 [G, K, N]: the fused gated
    up projection of an expert layer (zeros past the sum)."""
    import torch
    m, k = lhs.shape
    g, _, n = w0.shape
    out_dtype = out_dtype or lhs.dtype
    if out is not None:
        _check_out(out, m * n, out_dtype, lhs.device)
    names = {torch.bfloat16: "bf16", torch.float32: "f32"}
    s = _run_stream(stream, lhs.device)
    key = ("gated", m, k, n, g, out_dtype, lhs.device)
    plan, ws = _cached_plan(key, s, m=m, k=k, n=n, groups=g, mode="forward_gated", in_dtype="bf16",
                            out_dtype=names[out_dtype], device=lhs.device)
    with torch.cuda.stream(s):
        if out is None:
            out = torch.empty((m, n), dtype=out_dtype, device=lhs.device)
        rdot_forward_gated(plan.handle, lhs.contiguous(), w0.contiguous(), w1.contiguous(),
                           group_sizes.to(torch.int32).contiguous(), out, ws, s)
    return out


def grad_weight_mxfp8(lhs_q, lhs_s, dy_q, dy_s, group_sizes, out=None, stream=None, out_dtype=None):
    """MXFP8 weight gradient: ``dw [G, K, N]`` (fp32 by default, or bf16) from E4M3 codes with E8M0
    scales along the rows in blocks of 32 that start at each group's first row (scale tensors
    ``[M // 32 + G, K | N]``)."""
    import torch
    m, k = lhs_q.shape
    n = dy_q.shape[1]
    g = group_sizes.shape[0]
    out_dtype = out_dtype or (out.dtype if out is not None else torch.float32)
    if out is not None:
        _check_out(out, g * k * n, out_dtype, lhs_q.device)
    names = {torch.bfloat16: "bf16", torch.float32: "f32"}
    s = _run_stream(stream, lhs_q.device)
    key = ("wgrad_mxfp8", m, k, n, g, out_dtype, lhs_q.device)
    plan, ws = _cached_plan(key, s, m=m, k=k, n=n, groups=g, mode="grad_weight_mxfp8", in_dtype="e4m3",
                            out_dtype=names[out_dtype], device=lhs_q.device)
    with torch.cuda.stream(s):
        if out is None:
            out = torch.empty((g, k, n), dtype=out_dtype, device=lhs_q.device)
        rdot_grad_weight_mxfp8(plan.handle, lhs_q.contiguous(), lhs_s.contiguous(), dy_q.contiguous(),
                               dy_s.contiguous(), group_sizes.to(torch.int32).contiguous(), out, ws, s)
    return out


def ragged_dot_combine(lhs, rhs, group_sizes, order, topk_weights, out=None, stream=None):
    """``out[t] = sum_j w[t, j] * (lhs @ rhs[g])[inv[t*k + j]]`` in one pass (fp32 [T, N]): the down
    projection over the permuted rows with the weighted un-permute fused into its epilogue."""
    import torch
    m, kdim = lhs.shape
    g, _, n = rhs.shape
    t, k = topk_weights.shape
    if out is not None:
        _check_out(out, t * n, torch.float32, lhs.device)
    s = _run_stream(stream, lhs.device)
    key = ("fwd", m, kdim, n, g, "bf16", torch.float32, lhs.device)     # the fp32-out forward's plan
    plan, ws = _cached_plan(key, s, m=m, k=kdim, n=n, groups=g, mode="forward", in_dtype="bf16", out_dtype="f32",
                            device=lhs.device)
    with torch.cuda.stream(s):
        if out is None:
            out = torch.empty((t, n), dtype=torch.float32, device=lhs.device)
        rdot_forward_combine(plan.handle, lhs.contiguous(), rhs.contiguous(), group_sizes.to(torch.int32).contiguous(),
                             order.to(torch.int32).contiguous(), topk_weights.to(torch.float32).contiguous(), out,
                             ws, s)
    return out


def router_topk(logits, k, weights="softmax_topk", stream=None):
    """Each token's top-k experts and their weights: returns ``(ids int32 [T, k], w fp32 [T, k])``.
    ``weights``: "values" (the logits), "softmax" (over all experts) or "softmax_topk" (over the k)."""
    import torch
    s = _run_stream(stream, logits.device)
    with torch.cuda.stream(s):
        logits = logits.contiguous()
        t = logits.shape[0]
        ids = torch.empty((t, k), dtype=torch.int32, device=logits.device)
        w = torch.empty((t, k), dtype=torch.float32, device=logits.device)
        rdot_router_topk(logits, k, _ROUTER_MODES[weights], ids, w, s)
    return ids, w


def moe_permute(topk_ids, x, n_experts, stream=None):
    """Sorts the token copies by expert: returns ``(x_sorted [T*k, K], group_sizes [E], order,
    inv)`` for int32 topk_ids [T, k] and x [T, K] (any dtype with 16-byte rows)."""
    import torch
    t, k = topk_ids.shape
    dev = x.device
    s = _run_stream(stream, dev)
    with torch.cuda.stream(s):
        ids = topk_ids.to(device=dev, dtype=torch.int32).contiguous()
        gs = torch.empty(n_experts, dtype=torch.int32, device=dev)
        order = torch.empty(t * k, dtype=torch.int32, device=dev)
        inv = torch.empty(t * k, dtype=torch.int32, device=dev)
        xs = torch.empty((t * k, x.shape[1]), dtype=x.dtype, device=dev)
        ws = torch.empty(rdot_moe_route_workspace_size(t, k, n_experts), dtype=torch.uint8, device=dev)
        rdot_moe_permute(ids, x.contiguous(), n_experts, gs, order, inv, xs, ws, s)
    return xs, gs, order, inv


def moe_unpermute(y_sorted, inv, topk_weights, out=None, stream=None):
    """``out[t] = sum_j w[t, j] * y_sorted[inv[t*k + j]]`` (bf16 [T, N])."""
    import torch
    t, _ = topk_weights.shape
    if out is not None:
        _check_out(out, t * y_sorted.shape[1], torch.bfloat16, y_sorted.device)
    s = _run_stream(stream, y_sorted.device)
    with torch.cuda.stream(s):
        if out is None:
            out = torch.empty((t, y_sorted.shape[1]), dtype=torch.bfloat16, device=y_sorted.device)
        rdot_moe_unpermute(y_sorted.contiguous(), inv, topk_weights.to(torch.float32).contiguous(), out, s)
    return out


def quantize_mxfp4(x, values=False, stream=None):
    """MXFP4 quantisation of x [rows, K] (fp32 or bf16) in blocks of 32 along K: returns ``(codes uint8
    [rows, K/2], scales uint8 [rows, K/32])``, and with ``values`` also the bf16 [rows, K] they stand for."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be [rows, K]")
    m, k = x.shape
    s = _run_stream(stream, x.device)
    with torch.cuda.stream(s):
        codes = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((m, k // 32), dtype=torch.uint8, device=x.device)
        v = torch.empty((m, k), dtype=torch.bfloat16, device=x.device) if values else None
        rdot_quantize_mxfp4(x.contiguous(), codes, scales, v, s)
    return (codes, scales, v) if values else (codes, scales)


def quantize_mxfp4_weight(w, values=False, stream=None):
    """MXFP4 quantisation of weights w [G, K, N] (fp32 or bf16) along K, laid out for
    :func:`ragged_dot_mxfp4`: returns ``(codes uint8 [G, N, K/2], scales uint8 [G, ceil(N/128), ceil(K/128),
    512])``, and with ``values`` also the bf16 [G, K, N] they stand for."""
    import torch
    if w.dim() != 3:
        raise ValueError("w must be [G, K, N]")
    g, k, n = w.shape
    s = _run_stream(stream, w.device)
    with torch.cuda.stream(s):
        codes = torch.empty((g, n, k // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((g, -(-n // 128), -(-k // 128), 512), dtype=torch.uint8, device=w.device)
        v = torch.empty((g, k, n), dtype=torch.bfloat16, device=w.device) if values else None
        rdot_quantize_mxfp4_weight(w.contiguous(), codes, scales, v, s)
    return (codes, scales, v) if values else (codes, scales)


def ragged_dot_mxfp4(lhs_q, lhs_scale, rhs_q, rhs_scale, group_sizes, out=None, stream=None):
    """MXFP4 forward: codes and scales of :func:`quantize_mxfp4` (lhs, M rows in group order) and of
    :func:`quantize_mxfp4_weight` (rhs); bf16 out [M, N], rows past ``sum(group_sizes)`` zero."""
    import torch
    m, kh = lhs_q.shape
    g, n, kh2 = rhs_q.shape
    k = 2 * kh
    if (kh2 != kh or group_sizes.shape != (g,) or lhs_scale.shape != (m, k // 32)
            or rhs_scale.shape != (g, -(-n // 128), -(-k // 128), 512)):
        raise ValueError("shape mismatch between lhs, rhs, their scales and group_sizes")
    if any(t.dtype != torch.uint8 for t in (lhs_q, lhs_scale, rhs_q, rhs_scale)):
        raise TypeError("codes and scales must be uint8")
    _same_device(lhs_q, lhs_scale, rhs_q, rhs_scale, group_sizes)
    if out is not None:
        if out.shape != (m, n):
            raise ValueError("out must be [M, N]")
        _check_out(out, m * n, torch.bfloat16, lhs_q.device)
    s = _run_stream(stream, lhs_q.device)
    key = ("mxfp4", m, k, n, g, lhs_q.device)
    plan, ws = _cached_plan(key, s, m=m, k=k, n=n, groups=g, mode="forward_mxfp4", in_dtype="e2m1", out_dtype="bf16",
                            device=lhs_q.device)
    with torch.cuda.stream(s):
        if out is None:
            out = torch.empty((m, n), dtype=torch.bfloat16, device=lhs_q.device)
        rdot_forward_mxfp4(plan.handle, lhs_q.contiguous(), lhs_scale.contiguous(), rhs_q.contiguous(),
                           rhs_scale.contiguous(), group_sizes.to(torch.int32).contiguous(), out, ws, s)
    return out


def moe_unpermute_grad(dout, y_sorted, order, inv, topk_weights, stream=None):
    """The gradient of :func:`moe_unpermute`: returns ``(dy_sorted bf16 [T*k, N], dw fp32 [T, k])`` for
    the combined rows' gradient dout bf16 [T, N], the expert outputs y_sorted bf16 [T*k, N] that the
    forward combined, and :func:`moe_permute`'s order and inv."""
    import torch
    t, k = topk_weights.shape
    if dout.dtype != torch.bfloat16 or y_sorted.dtype != torch.bfloat16:
        raise TypeError("dout and y_sorted must be bfloat16")
    if dout.shape != (t, y_sorted.shape[1]) or y_sorted.shape[0] != t * k or order.numel() != t * k or inv.numel() != t * k:
        raise ValueError("shape mismatch between dout, y_sorted, order, inv and topk_weights")
    _same_device(dout, y_sorted, order, inv, topk_weights)
    s = _run_stream(stream, dout.device)
    with torch.cuda.stream(s):
        dy = torch.empty_like(y_sorted, memory_format=torch.contiguous_format)
        dw = torch.empty((t, k), dtype=torch.float32, device=dout.device)
        rdot_moe_unpermute_grad(dout.contiguous(), y_sorted.contiguous(), order.to(torch.int32).contiguous(),
                                inv.to(torch.int32).contiguous(), topk_weights.to(torch.float32).contiguous(), dy, dw, s)
    return dy, dw


def moe_permute_grad(dx_sorted, inv, k, stream=None):
    """The gradient of :func:`moe_permute`'s gather: dx [T, N] with ``dx[t]`` the sum of the rows of
    dx_sorted [T*k, N] (fp32 or bf16) that token t's kept copies were sorted to."""
    import torch
    if k < 1 or dx_sorted.dim() != 2 or dx_sorted.shape[0] % k or inv.numel() != dx_sorted.shape[0]:
        raise ValueError("dx_sorted must have T*k rows and inv T*k elements")
    _same_device(dx_sorted, inv)
    s = _run_stream(stream, dx_sorted.device)
    with torch.cuda.stream(s):
        dx = torch.empty((dx_sorted.shape[0] // k, dx_sorted.shape[1]), dtype=dx_sorted.dtype, device=dx_sorted.device)
        rdot_moe_permute_grad(dx_sorted.contiguous(), inv.to(torch.int32).contiguous(), dx, s)
    return dx


def router_topk_grad(logits, topk_ids, topk_weights, dweights, weights="softmax_topk", stream=None):
    """The gradient of :func:`router_topk`: dlogits (the logits' shape and dtype, fp32 or bf16) from the
    weights' gradient dweights [T, k]."""
    import torch
    t, _ = logits.shape
    if topk_ids.shape != topk_weights.shape or topk_ids.shape != dweights.shape or topk_ids.shape[0] != t:
        raise ValueError("topk_ids, topk_weights and dweights must all be [T, k]")
    _same_device(logits, topk_ids, topk_weights, dweights)
    s = _run_stream(stream, logits.device)
    with torch.cuda.stream(s):
        dlogits = torch.empty_like(logits, memory_format=torch.contiguous_format)
        rdot_router_topk_grad(logits.contiguous(), topk_ids.to(torch.int32).contiguous(),
                              topk_weights.to(torch.float32).contiguous(), dweights.to(torch.float32).contiguous(),
                              _ROUTER_MODES[weights], dlogits, s)
    return dlogits


def ragged_dot_mxfp8(lhs_q, lhs_scale, rhs_q, rhs_scale, group_sizes, out=None, stream=None):
    """MXFP8 forward: E4M3 codes (uint8) with E8M0 scales per 32 K elements; bf16 out."""
    import torch
    m, k = lhs_q.shape
    g, _, n = rhs_q.shape
    if out is not None:
        _check_out(out, m * n, torch.bfloat16, lhs_q.device)
    s = _run_stream(stream, lhs_q.device)
    key = ("mxfp8", m, k, n, g, lhs_q.device)
    plan, ws = _cached_plan(key, s, m=m, k=k, n=n, groups=g, mode="forward_mxfp8", in_dtype="e4m3", out_dtype="bf16",
                            device=lhs_q.device)
    with torch.cuda.stream(s):
        if out is None:
            out = torch.empty((m, n), dtype=torch.bfloat16, device=lhs_q.device)
        rdot_forward_mxfp8(plan.handle, lhs_q, lhs_scale, rhs_q, rhs_scale, group_sizes.to(torch.int32).contiguous(),
                           out, ws, s)
    return out


def padded_ragged_dot(lhs, rhs, group_sizes, capacity, out=None, pad_workspace=None, stream=None):
    """The padded-dense baseline: pad every group to ``capacity`` rows, one uniform batched GEMM,
    gather back. Returns ``(out, pad_workspace)`` so callers can reuse the scratch."""
    import torch
    m, k = lhs.shape
    g, _, n = rhs.shape
    if out is not None:
        _check_out(out, m * n, torch.bfloat16, lhs.device)
    s = _run_stream(stream, lhs.device)
    key = ("fwd", m, k, n, g, "bf16", torch.bfloat16, lhs.device)
    plan, ws = _cached_plan(key, s, m=m, k=k, n=n, groups=g, mode="forward", in_dtype="bf16", out_dtype="bf16",
                            device=lhs.device)
    need = rdot_padded_workspace_size(plan.handle, capacity)
    with torch.cuda.stream(s):
        if pad_workspace is None or pad_workspace.numel() < need:
            pad_workspace = torch.empty(need, dtype=torch.uint8, device=lhs.device)
        if out is None:
            out = torch.empty((m, n), dtype=torch.bfloat16, device=lhs.device)
        rdot_padded_forward(plan.handle, lhs, rhs, group_sizes.to(torch.int32).contiguous(), out, capacity,
                            pad_workspace, ws, s)
    return out, pad_workspace
