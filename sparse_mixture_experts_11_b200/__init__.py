"""Python binding of ``libmoe.so``, the sparse MoE layer forward pass on B200 (sm_100a).

The functions mirror the C ABI in ``include/moe.h`` name for name (without the ``moe_``
prefix). They only marshal arguments: they check torch tensors' dtype, shape, device and
contiguity, then pass raw device pointers and the current CUDA stream to the library. Every
step of the layer runs in the library's CUDA kernels. There is no fallback: importing this
package fails if the library is missing.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python sparse_mixture_experts_11_b200/build.py` "
        "(the MoE layer has no implementation other than this CUDA library)")
_lib = ctypes.CDLL(LIB_PATH)

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT, ERR_BOUNDS = 0, -1, -2, -3, -4, -5, -6
ACT_SWIGLU, ACT_GELU = 0, 1
_ACTS = {"swiglu": ACT_SWIGLU, "gelu": ACT_GELU}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class Dims(ctypes.Structure):
    """``moe_dims``: T, d_model, n_experts, top_k, d_ff, act, capacity."""
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("act", ctypes.c_int32),
                ("capacity", ctypes.c_int32)]

    def __repr__(self):
        return ("Dims(T={0.T}, d_model={0.d_model}, n_experts={0.n_experts}, top_k={0.top_k}, "
                "d_ff={0.d_ff}, act={0.act}, capacity={0.capacity})".format(self))


class ForwardBuffers(ctypes.Structure):
    """``moe_forward_buffers``: device pointers into a moe_forward workspace."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "logits", "topk_idx", "topk_w", "slot", "expert_count", "expert_offset", "row_of_pair",
        "pair_of_row", "x_perm", "h", "y_perm", "stage_ws")] + [("stage_ws_bytes", ctypes.c_size_t)]


WFMT_BF16, WFMT_MXFP8, WFMT_MXFP4, WFMT_MXFP8_BS, WFMT_MXFP4_BS = 0, 1, 2, 3, 4
# "_bs": the same weights on the block-scaled MMA, with MXFP8-quantised token rows and h
_WFMT = {"mxfp8": WFMT_MXFP8, "mxfp4": WFMT_MXFP4, "mxfp8_bs": WFMT_MXFP8_BS,
         "mxfp4_bs": WFMT_MXFP4_BS}


class MxWeights(ctypes.Structure):
    """``moe_mx_weights``: expert weights in an MX format (device pointers)."""
    _fields_ = [("fmt", ctypes.c_int32), ("gate_up", ctypes.c_void_p),
                ("gate_up_scales", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("down_scales", ctypes.c_void_p)]


ADAMW_BLOCK = 128  # MOE_ADAMW_BLOCK: elements that share a scale of 8-bit moments
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}  # moe_dtype


class GradTensor(ctypes.Structure):
    """``moe_grad_tensor``: one gradient of moe_grad_norm."""
    _fields_ = [("grad", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class AdamWTensor(ctypes.Structure):
    """``moe_adamw_tensor``: one tensor of moe_adamw_step."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("numel", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
        ("state_bits", ctypes.c_int32), ("weight_decay", ctypes.c_float)]


class AdamWConfig(ctypes.Structure):
    """``moe_adamw_config``: hyper-parameters of a step."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps")] + [
        ("step", ctypes.c_int32), ("seed", ctypes.c_uint32), ("step_dev", ctypes.c_void_p),
        ("lr_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p)]


_P = ctypes.c_void_p
_DIMS = ctypes.POINTER(Dims)
_MXW = ctypes.POINTER(MxWeights)
_SIGS = {
    "moe_capacity": (ctypes.c_int32, [ctypes.c_double, ctypes.c_int32, ctypes.c_int32]),
    "moe_max_rows": (ctypes.c_int64, [_DIMS]),
    "moe_workspace_bytes": (ctypes.c_int, [_DIMS, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_workspace_init": (ctypes.c_int, [_P, ctypes.c_size_t, _P]),
    "moe_route": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_route_from_logits": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_route_with_stats": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_float,
                                            _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_redirect_overflow": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_permute": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_grouped_ffn": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_unpermute_combine": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, ctypes.c_int32, _P,
                                             ctypes.c_size_t, _P]),
    "moe_forward_workspace_bytes": (ctypes.c_int, [_DIMS, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_mx_act_workspace_bytes": (ctypes.c_int, [_DIMS, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_forward_layout": (ctypes.c_int, [_DIMS, _P, ctypes.c_size_t, ctypes.POINTER(ForwardBuffers)]),
    "moe_forward": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_route_noalloc": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_grouped_ffn_mx": (ctypes.c_int, [_DIMS, _P, _P, _MXW, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_forward_mx": (ctypes.c_int, [_DIMS, _P, _P, _P, _MXW, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_router_stats": (ctypes.c_int, [_DIMS, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P,
                                        ctypes.c_size_t, _P]),
    "moe_backward_workspace_bytes": (ctypes.c_int, [_DIMS, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_backward": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P, _P, _P,
                                    _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_balance_loss": (ctypes.c_int, [_DIMS, _P, _P, _P, ctypes.c_float, ctypes.c_float, _P, _P, _P,
                                        _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_router_backward_workspace_bytes": (ctypes.c_int, [_DIMS, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_router_backward": (ctypes.c_int, [_DIMS, _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P,
                                           ctypes.c_size_t, _P]),
    "moe_grad_norm_workspace_bytes": (ctypes.c_int, [ctypes.POINTER(ctypes.c_size_t)]),
    "moe_grad_norm": (ctypes.c_int, [ctypes.POINTER(GradTensor), ctypes.c_int32, ctypes.c_float, _P, _P,
                                     _P, ctypes.c_size_t, _P]),
    "moe_adamw_step": (ctypes.c_int, [ctypes.POINTER(AdamWTensor), ctypes.c_int32,
                                      ctypes.POINTER(AdamWConfig), _P]),
    "moe_read_device_error": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int)]),
    "moe_debug_set_wait_timeout_ns": (ctypes.c_uint64, [ctypes.c_uint64]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


# ----------------------------------------------------------------------------- marshalling
def _check(status: int, where: str) -> None:
    if status != OK:
        raise MoeError(status, where)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # no Stream object made


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, shape=None, allow_none=False):
    if (t is not None and t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype is dtype)
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


# ----------------------------------------------------------------------------- host helpers
def debug_set_wait_timeout_ns(ns: int) -> int:
    """Limit of the kernels' bounded waits for later calls (0 = default 2 s); returns the old one."""
    return int(_lib.moe_debug_set_wait_timeout_ns(int(ns)))


def status_string(status: int) -> str:
    return _lib.moe_status_string(int(status)).decode()


def capacity(capacity_factor: Optional[float], T: int, n_experts: int) -> int:
    """ceil(capacity_factor * T / n_experts); None / <=0 / inf means no limit (T)."""
    cf = 0.0 if capacity_factor is None else float(capacity_factor)
    return int(_lib.moe_capacity(cf, int(T), int(n_experts)))


def make_dims(T: int, d_model: int, n_experts: int, top_k: int, d_ff: int, act="swiglu",
              capacity: Optional[int] = None) -> Dims:
    a = _ACTS[act] if isinstance(act, str) else int(act)
    return Dims(int(T), int(d_model), int(n_experts), int(top_k), int(d_ff), a,
                int(T if capacity is None else capacity))


def max_rows(dims: Dims) -> int:
    r = int(_lib.moe_max_rows(ctypes.byref(dims)))
    if r < 0:
        raise MoeError(ERR_INVALID, "moe_max_rows")
    return r


def workspace_bytes(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)), "moe_workspace_bytes")
    return int(n.value)


def forward_workspace_bytes(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_forward_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)),
           "moe_forward_workspace_bytes")
    return int(n.value)


def mx_act_workspace_bytes(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_mx_act_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)),
           "moe_mx_act_workspace_bytes")
    return int(n.value)


def new_workspace(dims: Dims, device=None, forward: bool = False,
                  block_scaled: bool = False) -> torch.Tensor:
    """A zeroed uint8 workspace tensor for the per-stage calls (or for moe_forward); with
    block_scaled, room for the block-scaled MX formats' quantised activations after it."""
    n = forward_workspace_bytes(dims) if forward else workspace_bytes(dims)
    if block_scaled:
        n = (n + 255) // 256 * 256 + mx_act_workspace_bytes(dims)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def forward_layout(dims: Dims, ws: torch.Tensor) -> ForwardBuffers:
    b = ForwardBuffers()
    _check(_lib.moe_forward_layout(ctypes.byref(dims), _ptr(ws, "ws", torch.uint8), _nbytes(ws),
                                   ctypes.byref(b)), "moe_forward_layout")
    return b


def read_device_error(ws: torch.Tensor, stream=None, offset_bytes: int = 0) -> int:
    err = ctypes.c_int(0)
    p = ctypes.c_void_p(ws.data_ptr() + offset_bytes)
    _check(_lib.moe_read_device_error(p, _stream(stream), ctypes.byref(err)), "moe_read_device_error")
    return int(err.value)


# ----------------------------------------------------------------------------- stages
def route(dims: Dims, x, w_router, logit_bias, logits, topk_idx, topk_w, slot, expert_count,
          ws, stream=None) -> None:
    T, d, N, k = dims.T, dims.d_model, dims.n_experts, dims.top_k
    _check(_lib.moe_route(
        ctypes.byref(dims), _ptr(x, "x", torch.bfloat16, (T, d)),
        _ptr(w_router, "w_router", torch.float32, (N, d)),
        _ptr(logit_bias, "logit_bias", torch.float32, (N,), allow_none=True),
        _ptr(logits, "logits", torch.float32, (T, N)), _ptr(topk_idx, "topk_idx", torch.int32, (T, k)),
        _ptr(topk_w, "topk_w", torch.float32, (T, k)), _ptr(slot, "slot", torch.int32, (T, k)),
        _ptr(expert_count, "expert_count", torch.int32, (N,)), _ptr(ws, "ws", torch.uint8),
        _nbytes(ws), _stream(stream)), "moe_route")


def route_noalloc(dims: Dims, x, w_router, logit_bias, logits, topk_idx, topk_w, slot,
                  expert_count, stream=None) -> None:
    """moe_route without a workspace argument: for callers that cannot allocate device memory.
    Its scratch is a fixed array inside the library, shared by all calls. Calls that overlap
    on the GPU race on it, and shapes beyond its size are rejected (MOE_ERR_WORKSPACE)."""
    T, d, N, k = dims.T, dims.d_model, dims.n_experts, dims.top_k
    _check(_lib.moe_route_noalloc(
        ctypes.byref(dims), _ptr(x, "x", torch.bfloat16, (T, d)),
        _ptr(w_router, "w_router", torch.float32, (N, d)),
        _ptr(logit_bias, "logit_bias", torch.float32, (N,), allow_none=True),
        _ptr(logits, "logits", torch.float32, (T, N)), _ptr(topk_idx, "topk_idx", torch.int32, (T, k)),
        _ptr(topk_w, "topk_w", torch.float32, (T, k)), _ptr(slot, "slot", torch.int32, (T, k)),
        _ptr(expert_count, "expert_count", torch.int32, (N,)), _stream(stream)), "moe_route_noalloc")


def route_with_stats(dims: Dims, x, w_router, logit_bias, logits, topk_idx, topk_w, slot,
                     expert_count, picks, prob_mean, aux_loss, dropped, ws, alpha=0.01,
                     stream=None) -> None:
    """moe_route with the router statistics emitted by the routing launches."""
    T, d, N, k = dims.T, dims.d_model, dims.n_experts, dims.top_k
    _check(_lib.moe_route_with_stats(
        ctypes.byref(dims), _ptr(x, "x", torch.bfloat16, (T, d)),
        _ptr(w_router, "w_router", torch.float32, (N, d)),
        _ptr(logit_bias, "logit_bias", torch.float32, (N,), allow_none=True),
        _ptr(logits, "logits", torch.float32, (T, N)), _ptr(topk_idx, "topk_idx", torch.int32, (T, k)),
        _ptr(topk_w, "topk_w", torch.float32, (T, k)), _ptr(slot, "slot", torch.int32, (T, k)),
        _ptr(expert_count, "expert_count", torch.int32, (N,)), ctypes.c_float(alpha),
        _ptr(picks, "picks", torch.int32, (N,)), _ptr(prob_mean, "prob_mean", torch.float32, (N,)),
        _ptr(aux_loss, "aux_loss", torch.float32, (1,)), _ptr(dropped, "dropped", torch.int32, (1,)),
        _ptr(ws, "ws", torch.uint8), _nbytes(ws), _stream(stream)), "moe_route_with_stats")


def route_from_logits(dims: Dims, logits, topk_idx, topk_w, slot, expert_count, ws,
                      stream=None) -> None:
    T, N, k = dims.T, dims.n_experts, dims.top_k
    _check(_lib.moe_route_from_logits(
        ctypes.byref(dims), _ptr(logits, "logits", torch.float32, (T, N)),
        _ptr(topk_idx, "topk_idx", torch.int32, (T, k)), _ptr(topk_w, "topk_w", torch.float32, (T, k)),
        _ptr(slot, "slot", torch.int32, (T, k)), _ptr(expert_count, "expert_count", torch.int32, (N,)),
        _ptr(ws, "ws", torch.uint8), _nbytes(ws), _stream(stream)), "moe_route_from_logits")


REDIRECT_MAX_PAIRS = 163840  # T * k limit of moe_redirect_overflow


def redirect_overflow(dims: Dims, logits, topk_idx, slot, expert_count, ws, stream=None) -> None:
    """Overflow policy "redirect" after route(): topk_idx is rewritten with the serving expert."""
    T, N, k = dims.T, dims.n_experts, dims.top_k
    _check(_lib.moe_redirect_overflow(
        ctypes.byref(dims), _ptr(logits, "logits", torch.float32, (T, N)),
        _ptr(topk_idx, "topk_idx", torch.int32, (T, k)), _ptr(slot, "slot", torch.int32, (T, k)),
        _ptr(expert_count, "expert_count", torch.int32, (N,)),
        _ptr(ws, "ws", torch.uint8), _nbytes(ws), _stream(stream)), "moe_redirect_overflow")


def permute(dims: Dims, x, topk_idx, slot, expert_count, expert_offset, row_of_pair,
            pair_of_row, x_perm, ws, stream=None) -> None:
    T, d, N, k = dims.T, dims.d_model, dims.n_experts, dims.top_k
    R = max_rows(dims)
    _check(_lib.moe_permute(
        ctypes.byref(dims), _ptr(x, "x", torch.bfloat16, (T, d)),
        _ptr(topk_idx, "topk_idx", torch.int32, (T, k)), _ptr(slot, "slot", torch.int32, (T, k)),
        _ptr(expert_count, "expert_count", torch.int32, (N,)),
        _ptr(expert_offset, "expert_offset", torch.int32, (N + 1,)),
        _ptr(row_of_pair, "row_of_pair", torch.int32, (T, k)),
        _ptr(pair_of_row, "pair_of_row", torch.int32, (R,)),
        _ptr(x_perm, "x_perm", torch.bfloat16, (R, d)), _ptr(ws, "ws", torch.uint8), _nbytes(ws),
        _stream(stream)), "moe_permute")


def grouped_ffn(dims: Dims, x_perm, expert_offset, w_gate_up, w_down, h, y_perm, ws,
                stream=None) -> None:
    d, N, F = dims.d_model, dims.n_experts, dims.d_ff
    R = max_rows(dims)
    rows = 2 * F if dims.act == ACT_SWIGLU else F
    _check(_lib.moe_grouped_ffn(
        ctypes.byref(dims), _ptr(x_perm, "x_perm", torch.bfloat16, (R, d)),
        _ptr(expert_offset, "expert_offset", torch.int32, (N + 1,)),
        _ptr(w_gate_up, "w_gate_up", torch.bfloat16, (N, rows, d)),
        _ptr(w_down, "w_down", torch.bfloat16, (N, d, F)), _ptr(h, "h", torch.bfloat16, (R, F)),
        _ptr(y_perm, "y_perm", torch.float32, (R, d)), _ptr(ws, "ws", torch.uint8), _nbytes(ws),
        _stream(stream)), "moe_grouped_ffn")


def mx_weights(dims: Dims, fmt: str, gate_up, gate_up_scales, down, down_scales) -> MxWeights:
    """Check shapes and dtypes of MX expert weights and describe them for the C ABI.
    gate_up [N, rows, d_model or d_model/2] uint8, gate_up_scales [N, d_model/32, rows] uint8,
    down [N, d_model, d_ff or d_ff/2] uint8, down_scales [N, d_ff/32, d_model] uint8."""
    d, N, F = dims.d_model, dims.n_experts, dims.d_ff
    rows = 2 * F if dims.act == ACT_SWIGLU else F
    per = 1 if fmt.startswith("mxfp8") else 2
    return MxWeights(_WFMT[fmt],
                     _ptr(gate_up, "gate_up", torch.uint8, (N, rows, d // per)),
                     _ptr(gate_up_scales, "gate_up_scales", torch.uint8, (N, d // 32, rows)),
                     _ptr(down, "down", torch.uint8, (N, d, F // per)),
                     _ptr(down_scales, "down_scales", torch.uint8, (N, F // 32, d)))


def grouped_ffn_mx(dims: Dims, x_perm, expert_offset, w: MxWeights, h, y_perm, ws,
                   stream=None) -> None:
    d, N, F = dims.d_model, dims.n_experts, dims.d_ff
    R = max_rows(dims)
    _check(_lib.moe_grouped_ffn_mx(
        ctypes.byref(dims), _ptr(x_perm, "x_perm", torch.bfloat16, (R, d)),
        _ptr(expert_offset, "expert_offset", torch.int32, (N + 1,)), ctypes.byref(w),
        _ptr(h, "h", torch.bfloat16, (R, F)), _ptr(y_perm, "y_perm", torch.float32, (R, d)),
        _ptr(ws, "ws", torch.uint8), _nbytes(ws), _stream(stream)), "moe_grouped_ffn_mx")


def forward_mx_into(dims: Dims, x, w_router, logit_bias, w: MxWeights, residual, out, ws,
                    stream=None) -> None:
    """moe_forward_mx with caller-provided output and workspace (no allocation)."""
    T, d, N = dims.T, dims.d_model, dims.n_experts
    _check(_lib.moe_forward_mx(
        ctypes.byref(dims), _ptr(x, "x", torch.bfloat16, (T, d)),
        _ptr(w_router, "w_router", torch.float32, (N, d)),
        _ptr(logit_bias, "logit_bias", torch.float32, (N,), allow_none=True), ctypes.byref(w),
        _ptr(residual, "residual", torch.bfloat16, (T, d), allow_none=True),
        _ptr(out, "out", torch.bfloat16, (T, d)), _ptr(ws, "ws", torch.uint8), _nbytes(ws),
        _stream(stream)), "moe_forward_mx")


def unpermute_combine(dims: Dims, y_perm, row_of_pair, topk_w, residual, out, ws=None,
                      stream=None) -> None:
    T, d, k = dims.T, dims.d_model, dims.top_k
    R = max_rows(dims)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out must be bf16 or fp32")
    _check(_lib.moe_unpermute_combine(
        ctypes.byref(dims), _ptr(y_perm, "y_perm", torch.float32, (R, d)),
        _ptr(row_of_pair, "row_of_pair", torch.int32, (T, k)),
        _ptr(topk_w, "topk_w", torch.float32, (T, k)),
        _ptr(residual, "residual", torch.bfloat16, (T, d), allow_none=True),
        _ptr(out, "out", None, (T, d)), 1 if out.dtype == torch.float32 else 0,
        _ptr(ws, "ws", torch.uint8, allow_none=True), _nbytes(ws), _stream(stream)),
        "moe_unpermute_combine")


def router_stats(dims: Dims, logits, topk_idx, slot, picks, prob_mean, aux_loss, dropped, ws,
                 alpha: float = 1e-2, stream=None) -> None:
    """Per-expert picks and mean router probability, dropped pairs, and the auxiliary loss
    alpha * N * sum_e (picks_e / T) * P_e."""
    T, N, k = dims.T, dims.n_experts, dims.top_k
    _check(_lib.moe_router_stats(
        ctypes.byref(dims), _ptr(logits, "logits", torch.float32, (T, N)),
        _ptr(topk_idx, "topk_idx", torch.int32, (T, k)), _ptr(slot, "slot", torch.int32, (T, k)),
        float(alpha), _ptr(picks, "picks", torch.int32, (N,)),
        _ptr(prob_mean, "prob_mean", torch.float32, (N,)),
        _ptr(aux_loss, "aux_loss", torch.float32, (1,)), _ptr(dropped, "dropped", torch.int32, (1,)),
        _ptr(ws, "ws", torch.uint8), _nbytes(ws), _stream(stream)), "moe_router_stats")


def forward_into(dims: Dims, x, w_router, logit_bias, w_gate_up, w_down, residual, out, ws,
                 stream=None) -> None:
    """moe_forward with caller-provided output and workspace (no allocation)."""
    T, d, N, F = dims.T, dims.d_model, dims.n_experts, dims.d_ff
    rows = 2 * F if dims.act == ACT_SWIGLU else F
    _check(_lib.moe_forward(
        ctypes.byref(dims), _ptr(x, "x", torch.bfloat16, (T, d)),
        _ptr(w_router, "w_router", torch.float32, (N, d)),
        _ptr(logit_bias, "logit_bias", torch.float32, (N,), allow_none=True),
        _ptr(w_gate_up, "w_gate_up", torch.bfloat16, (N, rows, d)),
        _ptr(w_down, "w_down", torch.bfloat16, (N, d, F)),
        _ptr(residual, "residual", torch.bfloat16, (T, d), allow_none=True),
        _ptr(out, "out", torch.bfloat16, (T, d)), _ptr(ws, "ws", torch.uint8), _nbytes(ws),
        _stream(stream)), "moe_forward")


def forward(x: torch.Tensor, w_router: torch.Tensor, w_gate_up: torch.Tensor,
            w_down: torch.Tensor, *, top_k: int, act: str = "swiglu",
            capacity_factor: Optional[float] = None, logit_bias: Optional[torch.Tensor] = None,
            residual: Optional[torch.Tensor] = None, use_residual: bool = True,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The whole layer; allocates the output (and a workspace unless one is given).

    ``residual`` defaults to ``x`` (the layer returns x + MoE(x)); pass use_residual=False for
    the MoE part alone.
    """
    T, d = x.shape
    N = w_router.shape[0]
    F = w_down.shape[2]
    dims = make_dims(T, d, N, top_k, F, act, capacity(capacity_factor, T, N))
    if workspace is None:
        workspace = new_workspace(dims, x.device, forward=True)
    out = torch.empty((T, d), dtype=torch.bfloat16, device=x.device)
    res = (x if residual is None else residual) if use_residual else None
    forward_into(dims, x, w_router, logit_bias, w_gate_up, w_down, res, out, workspace)
    return out


def exported_symbols() -> list:
    """Names of the functions include/moe.h declares (parsed from the header)."""
    import re
    hdr = os.path.join(os.path.dirname(_HERE), "include", "moe.h")
    with open(hdr) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(moe_\w+)\s*\(", text, flags=re.M)))


# ----------------------------------------------------------------------------- backward
def backward_workspace_bytes(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_backward_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)),
           "moe_backward_workspace_bytes")
    return int(n.value)


def new_backward_workspace(dims: Dims, device=None) -> torch.Tensor:
    return torch.zeros(backward_workspace_bytes(dims), dtype=torch.uint8, device=device or "cuda")


def backward_into(dims: Dims, x, w_router, w_gate_up, w_down, fwd_ws, d_out, d_x, d_w_router,
                  d_logit_bias, d_w_gate_up, d_w_down, ws, stream=None) -> None:
    """moe_backward after moe_forward (whose workspace is fwd_ws) on the same inputs."""
    T, d, N, F = dims.T, dims.d_model, dims.n_experts, dims.d_ff
    rows = 2 * F if dims.act == ACT_SWIGLU else F
    _check(_lib.moe_backward(
        ctypes.byref(dims), _ptr(x, "x", torch.bfloat16, (T, d)),
        _ptr(w_router, "w_router", torch.float32, (N, d)),
        _ptr(w_gate_up, "w_gate_up", torch.bfloat16, (N, rows, d)),
        _ptr(w_down, "w_down", torch.bfloat16, (N, d, F)),
        _ptr(fwd_ws, "fwd_ws", torch.uint8), _nbytes(fwd_ws),
        _ptr(d_out, "d_out", torch.bfloat16, (T, d)), _ptr(d_x, "d_x", torch.float32, (T, d)),
        _ptr(d_w_router, "d_w_router", torch.float32, (N, d)),
        _ptr(d_logit_bias, "d_logit_bias", torch.float32, (N,), allow_none=True),
        _ptr(d_w_gate_up, "d_w_gate_up", torch.float32, (N, rows, d)),
        _ptr(d_w_down, "d_w_down", torch.float32, (N, d, F)),
        _ptr(ws, "ws", torch.uint8), _nbytes(ws), _stream(stream)), "moe_backward")


# ----------------------------------------------------------------------------- training
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _arg(t, here: int, name: str, dtype, shape) -> int:
    """Address of a tensor that must lie on the current device (the library launches there). One
    short test where all is well: the smallest calls cost little more than this."""
    if t is not None and t.get_device() == here and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    p = _ptr(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{here}") if p is not None else None


def _opt(t, here: int, name: str, dtype, shape):
    return None if t is None else _arg(t, here, name, dtype, shape)


def _workspace(ws, here: int) -> tuple:
    if ws is not None and ws.get_device() == here and ws.dtype is torch.uint8 and ws.is_contiguous():
        return ws.data_ptr(), ws.numel()
    return _arg(ws, here, "ws", torch.uint8, None if ws is None else tuple(ws.shape)), _nbytes(ws)


def _stream_on(stream, here: int) -> int:
    return _raw_stream(here) if stream is None and _raw_stream is not None else _stream(stream)


def balance_loss(dims: Dims, logits, topk_idx, token_mask, counts, n_tokens, prob_mean, loss,
                 d_logits, ws, alpha: float = 1e-2, z_coef: float = 0.0, d_loss=None,
                 stream=None) -> None:
    """Balance loss and router z-loss over the tokens whose token_mask (uint8, bool or None) is not 0,
    per-expert counts, and the gradient of the logits (d_logits may be None). loss [3] receives
    balance + z, balance, z; d_loss, a scalar tensor or None (1), is the total's gradient."""
    T, N, k = dims.T, dims.n_experts, dims.top_k
    if token_mask is not None and token_mask.dtype is torch.bool:
        token_mask = token_mask.view(torch.uint8)
    here, f32, i32 = _device(), torch.float32, torch.int32
    wp, wn = _workspace(ws, here)
    _check(_lib.moe_balance_loss(
        ctypes.byref(dims), _arg(logits, here, "logits", f32, (T, N)), _arg(topk_idx, here, "topk_idx", i32, (T, k)),
        _opt(token_mask, here, "token_mask", torch.uint8, (T,)), alpha, z_coef,
        _opt(d_loss, here, "d_loss", f32, () if d_loss is not None and d_loss.dim() == 0 else (1,)),
        _arg(counts, here, "counts", i32, (N,)), _arg(n_tokens, here, "n_tokens", i32, (1,)),
        _arg(prob_mean, here, "prob_mean", f32, (N,)), _arg(loss, here, "loss", f32, (3,)),
        _opt(d_logits, here, "d_logits", f32, (T, N)), wp, wn, _stream_on(stream, here)), "moe_balance_loss")


def router_backward_workspace_bytes(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_router_backward_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)),
           "moe_router_backward_workspace_bytes")
    return int(n.value)


def new_router_backward_workspace(dims: Dims, device=None) -> torch.Tensor:
    return torch.zeros(router_backward_workspace_bytes(dims), dtype=torch.uint8, device=device or "cuda")


def router_backward(dims: Dims, x, w_router, d_logits, d_x, d_w_router, d_logit_bias, ws,
                    accumulate: bool = False, stream=None) -> None:
    """Gradient of the linear router for a dense gradient of the logits; outputs (each may be
    None) are written, or added to with accumulate (after backward_into)."""
    T, d, N = dims.T, dims.d_model, dims.n_experts
    here, f32 = _device(), torch.float32
    wp, wn = _workspace(ws, here)
    _check(_lib.moe_router_backward(
        ctypes.byref(dims), _arg(x, here, "x", torch.bfloat16, (T, d)), _arg(w_router, here, "w_router", f32, (N, d)),
        _arg(d_logits, here, "d_logits", f32, (T, N)), _opt(d_x, here, "d_x", f32, (T, d)),
        _opt(d_w_router, here, "d_w_router", f32, (N, d)), _opt(d_logit_bias, here, "d_logit_bias", f32, (N,)),
        1 if accumulate else 0, wp, wn, _stream_on(stream, here)), "moe_router_backward")


class _Plan:
    """A host array of tensor descriptors, with the tensors it points at."""

    def __init__(self, kind, items, refs):
        self.array = (kind * max(1, len(items)))(*items)
        self.n = len(items)
        self.refs = refs
        devices = {t.device for r in refs for t in r if t is not None}
        if len(devices) > 1:
            raise ValueError(f"the tensors are on several devices: {sorted(map(str, devices))}")
        device = next(iter(devices), None)
        self.index = None if device is None else device.index

    def check(self, kind, here: int, maker: str) -> None:
        if self.array._type_ is not kind:
            raise ValueError(f"this call takes a plan of {maker}()")
        if self.index is not None and self.index != here:
            raise ValueError(f"the plan's tensors are on cuda:{self.index}, the current device is cuda:{here}")


def grad_plan(grads) -> _Plan:
    """Descriptors of gradients (fp32 or bf16 tensors of any shape) for grad_norm, made once for
    buffers that are filled again each step."""
    grads = list(grads)
    items = []
    for i, g in enumerate(grads):
        if g.dtype not in _DTYPES:
            raise ValueError(f"gradient {i} must be fp32 or bf16, got {g.dtype}")
        items.append(GradTensor(_ptr(g, f"gradient {i}"), g.numel(), _DTYPES[g.dtype]))
    return _Plan(GradTensor, items, [(g,) for g in grads])


def new_grad_norm_workspace(device=None) -> torch.Tensor:
    n = ctypes.c_size_t(0)
    _check(_lib.moe_grad_norm_workspace_bytes(ctypes.byref(n)), "moe_grad_norm_workspace_bytes")
    return torch.zeros(int(n.value), dtype=torch.uint8, device=device or "cuda")


def grad_norm(plan: _Plan, max_norm: float, norm, scale, ws, stream=None) -> None:
    """norm [1]: the global norm of the plan's gradients; scale [1]: min(1, max_norm / (norm +
    1e-6)), or NaN (adamw_step then leaves the step out) where the norm is not finite."""
    here = _device()
    plan.check(GradTensor, here, "grad_plan")
    wp, wn = _workspace(ws, here)
    _check(_lib.moe_grad_norm(plan.array, plan.n, max_norm, _arg(norm, here, "norm", torch.float32, (1,)),
                              _arg(scale, here, "scale", torch.float32, (1,)), wp, wn, _stream_on(stream, here)),
           "moe_grad_norm")


def new_adamw_state(param: torch.Tensor, bits: int = 32) -> dict:
    """Zeroed moments of a parameter: m and v (fp32, or E4M3 codes with m_scale and v_scale)."""
    n = param.numel()
    if bits == 32:
        return {"m": torch.zeros(n, dtype=torch.float32, device=param.device),
                "v": torch.zeros(n, dtype=torch.float32, device=param.device)}
    if bits != 8:
        raise ValueError("bits must be 32 or 8")
    blocks = -(-n // ADAMW_BLOCK)
    codes = lambda: torch.zeros(n, dtype=torch.uint8, device=param.device).view(torch.float8_e4m3fn)
    return {"m": codes(), "v": codes(),
            "m_scale": torch.zeros(blocks, dtype=torch.float32, device=param.device),
            "v_scale": torch.zeros(blocks, dtype=torch.float32, device=param.device)}


def adamw_tensor(param, grad, m, v, *, master=None, m_scale=None, v_scale=None,
                 weight_decay: float = 0.0) -> tuple:
    """One tensor of an AdamW plan: param fp32 or bf16, grad fp32 or bf16, m and v both fp32 or
    both float8_e4m3fn (codes of m and of sqrt(v), with m_scale and v_scale [ceil(numel / 128)]).
    master: fp32 master copy of a bf16 param. The shapes may differ as long as numel agrees."""
    n = param.numel()
    for name, t in (("param", param), ("grad", grad)):
        if t.dtype not in _DTYPES:
            raise ValueError(f"{name} must be fp32 or bf16, got {t.dtype}")
    if m.dtype != v.dtype or m.dtype not in (torch.float32, torch.float8_e4m3fn):
        raise ValueError(f"m and v must both be fp32 or both float8_e4m3fn, got {m.dtype} and {v.dtype}")
    if master is not None and param.dtype != torch.bfloat16:
        raise ValueError("master goes with a bf16 param")
    eight = m.dtype == torch.float8_e4m3fn
    if eight != (m_scale is not None) or eight != (v_scale is not None):
        raise ValueError("m_scale and v_scale go with 8-bit moments, and only with them")
    for name, t in (("grad", grad), ("m", m), ("v", v), ("master", master)):
        if t is not None and t.numel() != n:
            raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    blocks = (-(-n // ADAMW_BLOCK),)
    d = AdamWTensor(_ptr(param, "param"), _ptr(master, "master", torch.float32, allow_none=True),
                    _ptr(grad, "grad"), _ptr(m, "m"), _ptr(v, "v"),
                    _ptr(m_scale, "m_scale", torch.float32, blocks, allow_none=True),
                    _ptr(v_scale, "v_scale", torch.float32, blocks, allow_none=True), n,
                    _DTYPES[param.dtype], _DTYPES[grad.dtype], 8 if eight else 32, float(weight_decay))
    return d, (param, grad, m, v, master, m_scale, v_scale)


def adamw_plan(tensors) -> _Plan:
    """Descriptors of many tensors (from adamw_tensor) for adamw_step, made once and used for
    every step: the plan keeps the tensors alive and their addresses. Gradients must be in the same
    buffers every step (as backward_into fills them); tensors elsewhere need another plan."""
    tensors = list(tensors)
    return _Plan(AdamWTensor, [d for d, _ in tensors], [r for _, r in tensors])


def adamw_step(plan: _Plan, step, *, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, seed: int = 0,
               grad_scale=None, stream=None) -> None:
    """One AdamW step over the plan's tensors. step: the number of this step, from 1, or an int32
    tensor [1] read when the kernel runs; lr: a number or an fp32 tensor [1] read likewise;
    grad_scale: fp32 tensor [1] (from grad_norm) or None. A rate or scale on the device that is not
    finite, or a step below 1 there, leaves the step out."""
    here, f32 = _device(), torch.float32
    plan.check(AdamWTensor, here, "adamw_plan")
    step_t = step if isinstance(step, torch.Tensor) else None
    lr_t = lr if isinstance(lr, torch.Tensor) else None
    cfg = AdamWConfig(0.0 if lr_t is not None else lr, betas[0], betas[1], eps, 1 if step_t is not None else step,
                      seed & 0xFFFFFFFF, _opt(step_t, here, "step", torch.int32, (1,)), _opt(lr_t, here, "lr", f32, (1,)),
                      _opt(grad_scale, here, "grad_scale", f32, (1,)))
    _check(_lib.moe_adamw_step(plan.array, plan.n, ctypes.byref(cfg), _stream_on(stream, here)), "moe_adamw_step")
