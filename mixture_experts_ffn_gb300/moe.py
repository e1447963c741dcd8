"""Thin Python binding over libmoe.so (argument marshalling only).

Every function here has the name of the C entry point it calls, takes CUDA
tensors, allocates missing outputs and workspaces with torch, and calls the C
ABI on the current torch stream.  All arithmetic runs in the library's CUDA
kernels; there is no Python or CPU fallback, and every call raises if the
library is missing or the device is not a CUDA device.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_OVERLAP, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, \
    MOE_ERR_TIMEOUT, MOE_ERR_DEVICE, MOE_ERR_WORKSPACE = range(8)
MOE_F32, MOE_BF16, MOE_F16 = 0, 1, 2
MOE_SCORING_SOFTMAX, MOE_SCORING_SIGMOID, MOE_SCORING_SQRT_SOFTPLUS = 0, 1, 2
MOE_ACT_SILU_AND_MUL, MOE_ACT_SWIGLU, MOE_ACT_IDENTITY, MOE_ACT_GELU_AND_MUL = 0, 1, 2, 3
MOE_ACT_RELU, MOE_ACT_GELU, MOE_ACT_SILU = 4, 5, 6
MOE_STATUS_BYTES = 256
MOE_LAYOUT_PSUM, MOE_LAYOUT_PER_ROW, MOE_LAYOUT_MASKED = 0, 1, 2

MOE_MX_E4M3, MOE_MX_E2M1 = 0, 1
MOE_QUANT_NONE, MOE_QUANT_MX_E4M3, MOE_QUANT_E4M3_BLOCK128 = 0, 1, 2
_GATED = (MOE_ACT_SILU_AND_MUL, MOE_ACT_SWIGLU, MOE_ACT_GELU_AND_MUL)
# types that MX codes and scales are taken in: bytes, or the format's own
_E4M3 = (torch.float8_e4m3fn, torch.uint8, torch.int8)
_E2M1 = (torch.uint8, torch.int8, getattr(torch, "float4_e2m1fn_x2", torch.uint8))
_E8M0 = (getattr(torch, "float8_e8m0fnu", torch.uint8), torch.uint8, torch.int8)

# C entry points and their argument types (mirrors include/moe.h)
_vp, _i, _i64, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, \
    ctypes.c_size_t


class RouteParams(ctypes.Structure):
    _fields_ = [("top_k", ctypes.c_int32), ("scoring", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("num_expert_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float),
                ("local_expert_start", ctypes.c_int32), ("local_expert_count", ctypes.c_int32),
                ("route_scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class ActParams(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("swiglu_fusion", ctypes.c_int32),
                ("limit", ctypes.c_float), ("alpha", ctypes.c_float), ("beta", ctypes.c_float)]


_SIGNATURES = {
    "moe_route": [_vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp],
    "moe_permute": [_vp, _i, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_route_permute": [_vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                          _sz, _vp],
    "moe_permute_gather": [_vp, _i, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp],
    "moe_permute_align": [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_grouped_gemm": [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp],
    "moe_grouped_gemm_workspace_size": [_i, _i, _i],
    "moe_permute_align_workspace_size": [_i, _i, _i],
    "moe_grouped_gemm_act": [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp],
    "moe_grouped_gemm_act_split": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp,
                                   _vp, _sz, _vp],
    "moe_ffn_forward_split": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                              _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_grouped_gemm_act_gathered": [_vp, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                                      _vp, _vp, _sz, _vp],
    "moe_grouped_gemm_down": [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _sz, _vp],
    "moe_combine": [_vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _vp],
    "swiglu": [_vp, _vp, _i64, _i, _i, _i, _f, _f, _f, _vp, _vp],
    "moe_indexed_mlp": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp, _sz, _vp],
    "moe_ffn_forward": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp,
                        _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_ffn_forward_host": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                             _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_shared_expert_mlp": [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp],
    "moe_ffn_forward_local": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                              _vp, _vp, _vp, _sz, _vp],
    "moe_grouped_gemm_fp8_masked": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _sz, _vp],
    "moe_mx_quantize": [_vp, _i64, _i, _i64, _i, _i, _vp, _vp, _vp],
    "moe_mx_dequantize": [_vp, _vp, _i64, _i, _i, _i, _vp, _vp],
    "moe_add_rms_norm": [_vp, _vp, _vp, _i, _i, _i, _f, _i, _vp, _vp, _vp, _vp, _vp],
    "moe_grouped_gemm_mx": [_vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                            _vp, _vp, _vp, _sz, _vp],
    "moe_grouped_gemm_mx_workspace_size": [_i, _i, _i, _i],
    "moe_ffn_forward_mx": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                           _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_workspace_size_mx": [_i, _i, _i, _i, _i],
    "moe_combine_backward": [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp],
    "moe_permute_backward": [_vp, _vp, _i, _i, _i, _i, _vp, _vp],
    "moe_act_checkpoint": [_vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp],
    "moe_act_backward": [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp],
    "moe_grouped_gemm_dgrad": [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _sz, _vp],
    "moe_grouped_gemm_wgrad": [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp],
    "moe_grouped_gemm_wgrad_workspace_size": [_i, _i, _i, _i],
    "moe_route_backward": [_vp, _vp, _vp, _i, _i, _vp, _vp, _vp],
    "moe_shared_expert_workspace_size": [_i, _i, _i, _i],
    "moe_ffn_forward_shared": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp,
                               _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_workspace_size_shared": [_i, _i, _i, _i, _i, _i, _i],
    "moe_workspace_size": [_i, _i, _i, _i, _i, _i],
    "moe_workspace_size_host": [_i, _i, _i, _i, _i, _i],
    "moe_permute_workspace_size": [_i, _i],
    "moe_clear_status": [_vp, _vp],
    "moe_sync_status": [_vp, _vp],
    "moe_status_string": [_i],
    "moe_launch_count": [],
    "moe_set_gemm_simt": [_i],
    "moe_test_force_wait_timeout": [_i, ctypes.c_longlong],
    "moe_profile_report": [ctypes.c_char_p, _sz],
}
_RESTYPES = {"moe_workspace_size": _sz, "moe_permute_workspace_size": _sz,
             "moe_workspace_size_host": _sz, "moe_shared_expert_workspace_size": _sz,
             "moe_workspace_size_shared": _sz, "moe_permute_align_workspace_size": _sz,
             "moe_grouped_gemm_workspace_size": _sz, "moe_workspace_size_mx": _sz,
             "moe_grouped_gemm_mx_workspace_size": _sz,
             "moe_grouped_gemm_wgrad_workspace_size": _sz,
             "moe_status_string": ctypes.c_char_p, "moe_launch_count": ctypes.c_uint64}

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m mixture_experts_ffn_gb300.build`")
        lib = ctypes.CDLL(path)
        for name, args in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = _RESTYPES.get(name, ctypes.c_int)
        _lib = lib
    return _lib


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = load_library().moe_status_string(status).decode()
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # None: a CPU build of torch


def _stream_of(t: torch.Tensor) -> int:
    """Handle of the current stream of t's device (an integer; a tenth of the
    time that building a Stream object takes, which counts for calls of a few
    microseconds)."""
    return _raw_stream(t.device.index)


def _dtype(d: torch.dtype) -> int:
    if d == torch.bfloat16:
        return MOE_BF16
    if d == torch.float32:
        return MOE_F32
    if d == torch.float16:
        return MOE_F16
    raise TypeError(f"unsupported dtype {d}")


def _dt(t: torch.Tensor) -> int:
    return _dtype(t.dtype)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _fits(t, shape: tuple, size: int, what: str):
    """t (given by the caller, or None) has this shape, in elements of `size` bytes."""
    if t is not None and (t.shape != shape or t.element_size() != size):
        raise ValueError(f"{what} is {list(shape)} in elements of {size} bytes")


def _typed(t, dtype: torch.dtype, what: str):
    """t (given by the caller, or None) is of the type the library reads or writes there."""
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{what} takes {dtype}")


def _coded(t, types: tuple, what: str):
    """t (given by the caller, or None) holds codes or scales of one MX format."""
    if t is not None and t.dtype not in types:
        raise TypeError(f"{what} takes {types[0]} or bytes, not {t.dtype}")


def _on_gpu(t):
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors only")


def _cuda(*ts):
    for t in ts:
        if t is not None:
            _on_gpu(t)
            if not t.is_contiguous():
                raise ValueError("libmoe takes contiguous tensors only")


def _is_current(device) -> bool:
    return device.index == torch._C._cuda_getDevice()


def _together(first, *ts):
    """first and those of ts that are given: contiguous CUDA tensors of the current device."""
    _on_gpu(first)
    dev = first.device
    if not first.is_contiguous():
        raise ValueError("libmoe takes contiguous tensors only")
    for t in ts:
        if t is not None and not (t.is_contiguous() and t.device == dev):
            raise ValueError("the tensors of a call are contiguous and on one CUDA device")
    if not _is_current(dev):
        raise ValueError("the tensors of a call are on the current device")


def _asked(out, shape: tuple, dtype: torch.dtype, like, what: str, twin=None):
    """An output argument: True makes one (like twin, an input of this shape and type, where
    there is one: a fifth less time), False or None is none, a tensor is checked."""
    if out is True:
        return torch.empty(shape, dtype=dtype, device=like.device) if twin is None else \
            torch.empty_like(twin)
    if out is False or out is None:
        return None
    _together(like, out)
    _typed(out, dtype, what)
    _fits(out, shape, out.element_size(), what)
    return out


def _segments(seg_end):
    """Segment ends of at least one expert, or None."""
    if seg_end is not None:
        _typed(seg_end, torch.int32, "seg_end")
        if seg_end.numel() == 0:  # to the library an empty tensor is none
            raise ValueError("seg_end is [E]")


def _made(out, shape: tuple, dtype: torch.dtype, like, what: str, twin=None):
    """An output that every call has: True makes one, a tensor is checked."""
    if out is False or out is None:
        raise ValueError(f"{what} is True or the tensor to write")
    return _asked(out, shape, dtype, like, what, twin)


def _ws(nbytes: int, device) -> torch.Tensor:
    """A fresh workspace with a cleared status word (torch's caching allocator
    returns 512-byte aligned blocks)."""
    ws = torch.empty(max(nbytes, MOE_STATUS_BYTES), dtype=torch.uint8, device=device)
    ws[:MOE_STATUS_BYTES].zero_()
    return ws


def route_params(top_k, scoring="softmax", renormalize=True, num_expert_group=1, topk_group=1,
                 routed_scaling_factor=1.0, local_expert_start=0, local_expert_count=0,
                 route_scale=1.0) -> RouteParams:
    sc = {"softmax": MOE_SCORING_SOFTMAX, "sigmoid": MOE_SCORING_SIGMOID,
          "sqrt_softplus": MOE_SCORING_SQRT_SOFTPLUS}.get(scoring, scoring)
    return RouteParams(top_k, sc, int(bool(renormalize)), num_expert_group, topk_group,
                       routed_scaling_factor, local_expert_start, local_expert_count, route_scale,
                       MOE_F32)


def _rp(p: RouteParams, logits) -> RouteParams:
    """A copy of p whose MoERouter type T (logits and router_probs) is the
    logits tensor's dtype."""
    q = RouteParams.from_buffer_copy(p)
    q.dtype = _dt(logits)
    return q


def act_params(kind=MOE_ACT_SILU_AND_MUL, swiglu_fusion=2, limit=0.0, alpha=1.0,
               beta=0.0) -> ActParams:
    return ActParams(kind, swiglu_fusion, limit, alpha, beta)


# ----------------------------------------------------------------- entry points
def moe_workspace_size(T, H, F, E, K, dtype=MOE_BF16) -> int:
    return load_library().moe_workspace_size(T, H, F, E, K, dtype)


def moe_permute_workspace_size(M, E) -> int:
    return load_library().moe_permute_workspace_size(M, E)


def moe_route(logits, p: RouteParams, correction_bias=None, expert_ids=None, topk_weights=None,
              topk_ids=None, router_probs=None, weight_scale=None):
    """Router; returns (topk_weights, topk_ids, router_probs, weight_scale)."""
    lib = load_library()
    _cuda(logits, correction_bias, expert_ids)
    T, E = logits.shape
    dev = logits.device
    if topk_weights is None:
        topk_weights = torch.empty((T, p.top_k), dtype=torch.float32, device=dev)
    if topk_ids is None:
        topk_ids = torch.empty((T, p.top_k), dtype=torch.int32, device=dev)
    if p.local_expert_count > 0:
        if router_probs is None:
            router_probs = torch.empty((T, p.local_expert_count), dtype=logits.dtype, device=dev)
        if weight_scale is None:
            weight_scale = torch.empty((T,), dtype=torch.float32, device=dev)
    _check("moe_route", lib.moe_route(_p(logits), _p(correction_bias), _p(expert_ids), T, E,
                                      ctypes.byref(_rp(p, logits)), _p(topk_weights), _p(topk_ids),
                                      _p(router_probs), _p(weight_scale), _stream()))
    return topk_weights, topk_ids, router_probs, weight_scale


def moe_permute(topk_ids, E: int, hidden=None, ws=None, with_gather=True):
    """Returns dict(expert_input, seg_end, row_to_route, route_to_row, ws)."""
    lib = load_library()
    _cuda(topk_ids, hidden)
    T, K = topk_ids.shape
    M = T * K
    dev = topk_ids.device
    H = hidden.shape[1] if hidden is not None else 0
    dt = _dt(hidden) if hidden is not None else MOE_BF16
    xin = None
    if with_gather and hidden is not None:
        xin = torch.empty((M, H), dtype=hidden.dtype, device=dev)
    seg_end = torch.empty((E,), dtype=torch.int32, device=dev)
    r2r = torch.empty((M,), dtype=torch.int32, device=dev)
    route_to_row = torch.empty((M,), dtype=torch.int32, device=dev)
    need = lib.moe_permute_workspace_size(M, E)
    if ws is None:
        ws = _ws(need, dev)
    _check("moe_permute", lib.moe_permute(_p(hidden if xin is not None else None), dt,
                                          _p(topk_ids), T, H, E, K, _p(xin), _p(seg_end), _p(r2r),
                                          _p(route_to_row), _p(ws), ws.numel(), _stream()))
    return {"expert_input": xin, "seg_end": seg_end, "row_to_route": r2r,
            "route_to_row": route_to_row, "ws": ws}


def moe_grouped_gemm(a, w, layout: int, layout_metadata, N: int, act=None, bias=None, out=None,
                     ws=None):
    """The grouped GEMM over a row layout (MOE_LAYOUT_PSUM / PER_ROW: a [M, K],
    out [M, N]; MASKED: a [E, max_m, K], out [E, max_m, N]); w [E, N1, K]."""
    lib = load_library()
    _cuda(a, w, bias, layout_metadata)
    E, _, K = w.shape
    masked = layout == MOE_LAYOUT_MASKED
    rows = a.shape[1] if masked else a.shape[0]
    if out is None:
        shape = (E, rows, N) if masked else (rows, N)
        out = torch.empty(shape, dtype=a.dtype, device=a.device)
    if ws is None:
        ws = _ws(lib.moe_grouped_gemm_workspace_size(layout, rows, E), a.device)
    _check("moe_grouped_gemm",
           lib.moe_grouped_gemm(_p(a), _p(w), _p(bias), layout, _p(layout_metadata), rows, N, K, E,
                                _dt(a), None if act is None else ctypes.byref(act), _p(out),
                                _p(ws), ws.numel(), _stream()))
    return out


def moe_permute_align(topk_ids, E: int, block_size: int = 64, ws=None):
    """Padded layout: returns (sorted_token_ids, expert_ids, num_tokens_post_pad)."""
    lib = load_library()
    _cuda(topk_ids)
    T, K = topk_ids.shape
    dev = topk_ids.device
    L = T * K + (E + 1) * (block_size - 1)
    sorted_ids = torch.empty((L,), dtype=torch.int32, device=dev)
    expert_ids = torch.empty(((L + block_size - 1) // block_size,), dtype=torch.int32, device=dev)
    npp = torch.empty((1,), dtype=torch.int32, device=dev)
    if ws is None:
        ws = _ws(lib.moe_permute_align_workspace_size(T, K, E), dev)
    _check("moe_permute_align",
           lib.moe_permute_align(_p(topk_ids), T, K, E, block_size, _p(sorted_ids),
                                 _p(expert_ids), _p(npp), _p(ws), ws.numel(), _stream()))
    return sorted_ids, expert_ids, npp


def moe_permute_gather(hidden, seg_end, row_to_route, K: int, out=None, ws=None):
    """The permuted copy of the activations from index maps already built:
    out[row] = hidden[row_to_route[row] // K] for the rows below seg_end[-1]."""
    lib = load_library()
    _cuda(hidden, seg_end, row_to_route)
    T, H = hidden.shape
    E = seg_end.numel()
    if out is None:
        out = torch.empty((T * K, H), dtype=hidden.dtype, device=hidden.device)
    if ws is None:
        ws = _ws(MOE_STATUS_BYTES, hidden.device)
    _check("moe_permute_gather",
           lib.moe_permute_gather(_p(hidden), _dt(hidden), _p(seg_end), _p(row_to_route), T, H, E,
                                  K, _p(out), _p(ws), ws.numel(), _stream()))
    return out


def moe_route_permute(logits, p: RouteParams, correction_bias=None, expert_ids=None, ws=None):
    """moe_route then the index maps of moe_permute, in one launch; returns
    (topk_weights, topk_ids, router_probs, weight_scale, maps) with maps =
    dict(seg_end, row_to_route, route_to_row, ws)."""
    lib = load_library()
    _cuda(logits, correction_bias, expert_ids)
    T, E = logits.shape
    K = p.top_k
    dev = logits.device
    tw = torch.empty((T, K), dtype=torch.float32, device=dev)
    ti = torch.empty((T, K), dtype=torch.int32, device=dev)
    probs = wsc = None
    if p.local_expert_count > 0:
        probs = torch.empty((T, p.local_expert_count), dtype=logits.dtype, device=dev)
        wsc = torch.empty((T,), dtype=torch.float32, device=dev)
    seg_end = torch.empty((E,), dtype=torch.int32, device=dev)
    r2r = torch.empty((T * K,), dtype=torch.int32, device=dev)
    route_to_row = torch.empty((T * K,), dtype=torch.int32, device=dev)
    if ws is None:
        ws = _ws(lib.moe_permute_workspace_size(T * K, E), dev)
    _check("moe_route_permute",
           lib.moe_route_permute(_p(logits), _p(correction_bias), _p(expert_ids), T, E,
                                 ctypes.byref(_rp(p, logits)), _p(tw), _p(ti), _p(probs), _p(wsc),
                                 _p(seg_end),
                                 _p(r2r), _p(route_to_row), _p(ws), ws.numel(), _stream()))
    return tw, ti, probs, wsc, {"seg_end": seg_end, "row_to_route": r2r,
                                "route_to_row": route_to_row, "ws": ws}


def moe_grouped_gemm_act(a, w_gate_up, seg_end, F: int, act: ActParams, b_gate_up=None, out=None,
                         ws=None):
    lib = load_library()
    _cuda(a, w_gate_up, seg_end, b_gate_up)
    M, Hk = a.shape
    E = w_gate_up.shape[0]
    if out is None:
        out = torch.empty((M, F), dtype=a.dtype, device=a.device)
    if ws is None:
        ws = _ws(MOE_STATUS_BYTES, a.device)
    _check("moe_grouped_gemm_act",
           lib.moe_grouped_gemm_act(_p(a), _p(w_gate_up), _p(b_gate_up), _p(seg_end), M, F, Hk, E,
                                    _dt(a), ctypes.byref(act), _p(out), _p(ws), ws.numel(),
                                    _stream()))
    return out


def moe_grouped_gemm_act_split(a, w_gate, w_up, seg_end, act: ActParams, b_gate=None, b_up=None,
                               out=None, ws=None):
    """moe_grouped_gemm_act with the gate and up projections in two tensors
    w_gate, w_up [E, F, Hk] (SwiGLU fusion 0); returns out [M, F]."""
    lib = load_library()
    _cuda(a, w_gate, w_up, seg_end, b_gate, b_up)
    M, Hk = a.shape
    E, F, _ = w_gate.shape
    if out is None:
        out = torch.empty((M, F), dtype=a.dtype, device=a.device)
    if ws is None:
        ws = _ws(MOE_STATUS_BYTES, a.device)
    _check("moe_grouped_gemm_act_split",
           lib.moe_grouped_gemm_act_split(_p(a), _p(w_gate), _p(w_up), _p(b_gate), _p(b_up),
                                          _p(seg_end), M, F, Hk, E, _dt(a), ctypes.byref(act),
                                          _p(out), _p(ws), ws.numel(), _stream()))
    return out


def moe_grouped_gemm_act_gathered(hidden, row_to_route, top_k: int, w_gate_up, seg_end, F: int,
                                  act: ActParams, b_gate_up=None, out=None, ws=None):
    """moe_grouped_gemm_act with row m of the operand read as
    hidden[row_to_route[m] // top_k] (no permuted copy of the activations)."""
    lib = load_library()
    _cuda(hidden, row_to_route, w_gate_up, seg_end, b_gate_up)
    T, H = hidden.shape
    M = row_to_route.numel()
    E = w_gate_up.shape[0]
    if out is None:
        out = torch.empty((M, F), dtype=hidden.dtype, device=hidden.device)
    if ws is None:
        ws = _ws(MOE_STATUS_BYTES, hidden.device)
    _check("moe_grouped_gemm_act_gathered",
           lib.moe_grouped_gemm_act_gathered(_p(hidden), T, _p(row_to_route), top_k,
                                             _p(w_gate_up), _p(b_gate_up), _p(seg_end), M, F, H,
                                             E, _dt(hidden), ctypes.byref(act), _p(out), _p(ws),
                                             ws.numel(), _stream()))
    return out


def moe_grouped_gemm_down(a, w_down, seg_end, b_down=None, out=None, ws=None):
    lib = load_library()
    _cuda(a, w_down, seg_end, b_down)
    M, F = a.shape
    E, H, _ = w_down.shape
    if out is None:
        out = torch.empty((M, H), dtype=a.dtype, device=a.device)
    if ws is None:
        ws = _ws(MOE_STATUS_BYTES, a.device)
    _check("moe_grouped_gemm_down",
           lib.moe_grouped_gemm_down(_p(a), _p(w_down), _p(b_down), _p(seg_end), M, H, F, E,
                                     _dt(a), _p(out), _p(ws), ws.numel(), _stream()))
    return out


def moe_combine(expert_out, topk_weights, route_to_row, scale=1.0, out=None):
    lib = load_library()
    _cuda(expert_out, topk_weights, route_to_row)
    T, K = topk_weights.shape
    H = expert_out.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=expert_out.dtype, device=expert_out.device)
    _check("moe_combine", lib.moe_combine(_p(expert_out), _p(topk_weights), _p(route_to_row), T, K,
                                          H, _dt(expert_out), scale, _p(out), _stream()))
    return out


def swiglu(gate, up=None, swiglu_fusion=2, limit=0.0, alpha=1.0, beta=0.0, out=None):
    """The standalone SwiGLU op.  gate [R, 2I] (up None) or gate, up [R, I]."""
    lib = load_library()
    _cuda(gate, up)
    R = gate.shape[0]
    I = gate.shape[1] if up is not None else gate.shape[1] // 2
    if out is None:
        out = torch.empty((R, I), dtype=gate.dtype, device=gate.device)
    _check("swiglu", lib.swiglu(_p(gate), _p(up), R, I, _dt(gate), swiglu_fusion, limit, alpha,
                                beta, _p(out), _stream()))
    return out


def moe_indexed_mlp(hidden, w_gate_up, w_down, topk_weights, topk_ids, scale=1.0, out=None,
                    ws=None):
    lib = load_library()
    _cuda(hidden, w_gate_up, w_down, topk_weights, topk_ids)
    T, H = hidden.shape
    E, H2, F = w_down.shape
    K = topk_ids.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=hidden.dtype, device=hidden.device)
    if ws is None:
        ws = _ws(lib.moe_workspace_size(T, H, F, E, K, MOE_BF16), hidden.device)
    _check("moe_indexed_mlp",
           lib.moe_indexed_mlp(_p(hidden), _p(w_gate_up), _p(w_down), _p(topk_weights),
                               _p(topk_ids), T, H, F, E, K, scale, _p(out), _p(ws), ws.numel(),
                               _stream()))
    return out


def moe_ffn_forward(hidden, logits, w_gate_up, w_down, p: RouteParams, act: ActParams,
                    correction_bias=None, expert_ids=None, b_gate_up=None, b_down=None, out=None,
                    topk_weights_out=None, topk_ids_out=None, router_probs=None,
                    weight_scale=None, ws=None):
    """The whole routed MoE FFN forward; returns ``out`` [T, H]."""
    lib = load_library()
    _cuda(hidden, logits, w_gate_up, w_down, correction_bias, expert_ids, b_gate_up, b_down)
    T, H = hidden.shape
    E, _, F = w_down.shape
    if out is None:
        out = torch.empty_like(hidden)
    if ws is None:
        ws = _ws(lib.moe_workspace_size(T, H, F, E, p.top_k, _dt(hidden)), hidden.device)
    _check("moe_ffn_forward",
           lib.moe_ffn_forward(_p(hidden), _p(logits), _p(w_gate_up), _p(w_down),
                               _p(correction_bias), _p(expert_ids), _p(b_gate_up), _p(b_down), T,
                               H, F, E, _dt(hidden), ctypes.byref(_rp(p, logits)),
                               ctypes.byref(act), _p(out),
                               _p(topk_weights_out), _p(topk_ids_out), _p(router_probs),
                               _p(weight_scale), _p(ws), ws.numel(), _stream()))
    return out


def moe_ffn_forward_split(hidden, logits, w_gate, w_up, w_down, p: RouteParams, act: ActParams,
                          correction_bias=None, expert_ids=None, b_gate=None, b_up=None,
                          b_down=None, out=None, topk_weights_out=None, topk_ids_out=None,
                          router_probs=None, weight_scale=None, ws=None):
    """moe_ffn_forward with the gate and up projections in two tensors
    w_gate, w_up [E, F, H] (SwiGLU fusion 0); returns ``out`` [T, H]."""
    lib = load_library()
    _cuda(hidden, logits, w_gate, w_up, w_down, correction_bias, expert_ids, b_gate, b_up,
          b_down)
    T, H = hidden.shape
    E, _, F = w_down.shape
    if out is None:
        out = torch.empty_like(hidden)
    if ws is None:
        ws = _ws(lib.moe_workspace_size(T, H, F, E, p.top_k, _dt(hidden)), hidden.device)
    _check("moe_ffn_forward_split",
           lib.moe_ffn_forward_split(_p(hidden), _p(logits), _p(w_gate), _p(w_up), _p(w_down),
                                     _p(correction_bias), _p(expert_ids), _p(b_gate), _p(b_up),
                                     _p(b_down), T, H, F, E, _dt(hidden),
                                     ctypes.byref(_rp(p, logits)),
                                     ctypes.byref(act), _p(out), _p(topk_weights_out),
                                     _p(topk_ids_out), _p(router_probs), _p(weight_scale),
                                     _p(ws), ws.numel(), _stream()))
    return out


def moe_grouped_gemm_fp8_masked(a, a_scale, b, b_scale, layout_metadata, out=None, ws=None):
    """Block-scaled FP8 GEMM per expert over a masked slab: a [E, max_m, K] and
    b [E, N, K] float8_e4m3fn (or their uint8 codes), a_scale [E, max_m, K/128]
    and b_scale [E, N/128, K/128] float32, layout_metadata [E] int32 valid row
    counts; returns out [E, max_m, N] bf16 (rows past a count undefined)."""
    lib = load_library()
    _cuda(a, a_scale, b, b_scale, layout_metadata)
    E, max_m, K = a.shape
    N = b.shape[1]
    if out is None:
        out = torch.empty((E, max_m, N), dtype=torch.bfloat16, device=a.device)
    if ws is None:
        ws = _ws(MOE_STATUS_BYTES, a.device)
    _check("moe_grouped_gemm_fp8_masked",
           lib.moe_grouped_gemm_fp8_masked(_p(a), _p(a_scale), _p(b), _p(b_scale),
                                           _p(layout_metadata), E, max_m, N, K, _p(out), _p(ws),
                                           ws.numel(), _stream()))
    return out


def moe_mx_columns(K: int) -> int:
    """Columns of an MX row of K values: K rounded up to a multiple of 128."""
    return (K + 127) // 128 * 128


def moe_mx_quantize(x, format: int = MOE_MX_E4M3, codes=None, scales=None):
    """Rows of x [..., K] as microscaled floats: (codes, scales), codes [..., Kp]
    float8_e4m3fn or [..., Kp / 2] uint8 (MOE_MX_E2M1, two to a byte), scales
    [..., Kp / 32] float8_e8m0fnu, Kp = moe_mx_columns(K).  A 2-D x may have any
    row stride >= K; other shapes are contiguous."""
    lib = load_library()
    _on_gpu(x)
    K = x.shape[-1]
    if x.dim() == 2 and x.shape[0] > 1 and x.stride(1) == 1 and x.stride(0) >= K:
        stride = x.stride(0)
    elif x.is_contiguous():
        stride = K
    else:
        raise ValueError("moe_mx_quantize takes contiguous rows")
    Kp = moe_mx_columns(K)
    rows = x.numel() // K if K else 0
    lead, wide = x.shape[:-1], Kp // 2 if format == MOE_MX_E2M1 else Kp
    if codes is None:
        codes = torch.empty((*lead, wide), device=x.device,
                            dtype=torch.uint8 if format == MOE_MX_E2M1 else torch.float8_e4m3fn)
    else:
        _cuda(codes)
        _coded(codes, _E2M1 if format == MOE_MX_E2M1 else _E4M3, "codes")
        _fits(codes, (*lead, wide), 1, "codes")
    if scales is None:
        scales = torch.empty((*lead, Kp // 32), dtype=torch.float8_e8m0fnu, device=x.device)
    else:
        _cuda(scales)
        _coded(scales, _E8M0, "scales")
        _fits(scales, (*lead, Kp // 32), 1, "scales")
    _check("moe_mx_quantize",
           lib.moe_mx_quantize(x.data_ptr(), rows, K, stride, _dt(x), format, codes.data_ptr(),
                               scales.data_ptr(), _stream_of(x)))
    return codes, scales


def moe_mx_dequantize(codes, scales, K: int, format=None, dtype=torch.bfloat16, out=None):
    """The values of an MX tensor, [..., K] in dtype.  format defaults to the
    codes' own (MOE_MX_E2M1 when they are half as wide as an e4m3 row)."""
    lib = load_library()
    _cuda(codes, scales)
    if format is None:
        format = MOE_MX_E2M1 if codes.shape[-1] * 2 == scales.shape[-1] * 32 else MOE_MX_E4M3
    Kp = moe_mx_columns(K)
    if codes.shape[-1] != (Kp // 2 if format == MOE_MX_E2M1 else Kp) or \
            scales.shape[-1] * 32 != Kp or codes.shape[:-1] != scales.shape[:-1]:
        raise ValueError("codes and scales are not an MX tensor of K columns")
    rows = scales.numel() // (Kp // 32)
    _coded(codes, _E2M1 if format == MOE_MX_E2M1 else _E4M3, "codes")
    _coded(scales, _E8M0, "scales")
    if out is None:
        out = torch.empty((*codes.shape[:-1], K), dtype=dtype, device=codes.device)
    else:
        _cuda(out)
        _fits(out, (*codes.shape[:-1], K), out.element_size(), "out")
    _check("moe_mx_dequantize",
           lib.moe_mx_dequantize(codes.data_ptr(), scales.data_ptr(), rows, K, format, _dt(out),
                                 out.data_ptr(), _stream_of(codes)))
    return out


def moe_add_rms_norm(x, weight, residual=None, eps=1e-6, quant: int = MOE_QUANT_NONE, out=True,
                     residual_out=None, codes=None, scales=None):
    """h = x + residual (rounded; x without a residual), y = h * rsqrt(mean(h^2)
    + eps) * weight; returns dict(residual=h or None, out=y or None, codes,
    scales): y in 8 bits, MX (MOE_QUANT_MX_E4M3) or with a float32 scale per 128
    columns (MOE_QUANT_E4M3_BLOCK128).  out: True, False, or the tensor to
    write; residual_out may be residual itself."""
    lib = load_library()
    _cuda(x, weight, residual, residual_out, codes, scales)
    if weight.dtype != x.dtype or (residual is not None and residual.dtype != x.dtype):
        raise TypeError("x, weight and residual take one dtype")
    T, H = x.shape
    if weight.numel() != H or (residual is not None and residual.shape != x.shape):
        raise ValueError("weight is [H] and residual has the shape of x")
    if out is True:
        out = torch.empty_like(x)
    elif out is False:
        out = None
    else:
        _cuda(out)
        _typed(out, x.dtype, "out")
        _fits(out, x.shape, x.element_size(), "out")
    if residual_out is not None:
        _typed(residual_out, x.dtype, "residual_out")
        _fits(residual_out, x.shape, x.element_size(), "residual_out")
    elif residual is not None:
        residual_out = torch.empty_like(x)
    if quant != MOE_QUANT_NONE:
        Hp, mx = moe_mx_columns(H), quant == MOE_QUANT_MX_E4M3
        if codes is None:
            codes = torch.empty((T, Hp), dtype=torch.float8_e4m3fn, device=x.device)
        else:
            _coded(codes, _E4M3, "codes")
            _fits(codes, (T, Hp), 1, "codes")
        if scales is None:
            scales = torch.empty((T, Hp // (32 if mx else 128)), device=x.device,
                                 dtype=torch.float8_e8m0fnu if mx else torch.float32)
        else:
            _coded(scales, _E8M0 if mx else (torch.float32,), "scales")
            _fits(scales, (T, Hp // (32 if mx else 128)), 1 if mx else 4, "scales")
    _check("moe_add_rms_norm",
           lib.moe_add_rms_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), T, H, _dt(x), eps,
                                quant, _ptr(residual_out), _ptr(out), _ptr(codes), _ptr(scales),
                                _stream_of(x)))
    return {"residual": residual_out, "out": out, "codes": codes, "scales": scales}


def moe_grouped_gemm_mx_workspace_size(M, N, K, E) -> int:
    return load_library().moe_grouped_gemm_mx_workspace_size(M, N, K, E)


def moe_grouped_gemm_mx(a, a_scale, w, w_scale, seg_end, N: int, act: Optional[ActParams] = None,
                        bias=None, row_to_route=None, top_k: int = 1, dtype=torch.bfloat16,
                        mx_out: bool = False, out=None, out_scale=None, ws=None):
    """Grouped GEMM of MX e4m3 rows a [R, Kp] by MX e2m1 weights w [E, N1, Kp / 2]
    over the tight layout; row m is a[row_to_route[m] // top_k] when row_to_route
    is given.  Returns out [M, N] in dtype, or with mx_out the MX e4m3 rows
    (codes [M, Np], scales [M, Np / 32]).  dtype, the type of out and of the
    bias, is bfloat16, float16 or float32."""
    lib = load_library()
    _cuda(a, a_scale, w, w_scale, seg_end, bias, row_to_route, out, out_scale, ws)
    dt = _dtype(dtype)
    R, Kp = a.shape
    E, N1, half = w.shape
    M = R if row_to_route is None else row_to_route.numel()
    gated = act is not None and act.kind in _GATED
    if Kp % 128 or half * 2 != Kp or a_scale.shape != (R, Kp // 32) or \
            w_scale.shape != (E, N1, Kp // 32) or N1 != (2 * N if gated else N) or \
            seg_end.numel() != E or (bias is not None and bias.shape != (E, N1)):
        raise ValueError("operands are not MX tensors of matching extents")
    if bias is not None and bias.dtype != dtype:
        raise TypeError("bias takes the output's dtype")
    if a.dtype not in _E4M3 or a_scale.dtype not in _E8M0 or w.dtype not in _E2M1 or \
            w_scale.dtype not in _E8M0 or seg_end.dtype != torch.int32 or \
            (row_to_route is not None and row_to_route.dtype != torch.int32):
        raise TypeError("a is e4m3, w e2m1, the scales e8m0 (or bytes), seg_end and row_to_route int32")
    if mx_out:
        Np = moe_mx_columns(N)
        _coded(out, _E4M3, "out")
        _coded(out_scale, _E8M0, "out_scale")
        _fits(out, (M, Np), 1, "out")
        _fits(out_scale, (M, Np // 32), 1, "out_scale")
        if out is None:
            out = torch.empty((M, Np), dtype=torch.float8_e4m3fn, device=a.device)
        if out_scale is None:
            out_scale = torch.empty((M, Np // 32), dtype=torch.float8_e8m0fnu, device=a.device)
    elif out_scale is not None:  # to the library a scale buffer asks for MX rows
        raise ValueError("out_scale goes with mx_out")
    elif out is None:
        out = torch.empty((M, N), dtype=dtype, device=a.device)
    else:
        _typed(out, dtype, "out")
        _fits(out, (M, N), out.element_size(), "out")
    if ws is None:
        ws = _ws(lib.moe_grouped_gemm_mx_workspace_size(M, N, Kp, E), a.device)
    _check("moe_grouped_gemm_mx",
           lib.moe_grouped_gemm_mx(a.data_ptr(), a_scale.data_ptr(), R, _ptr(row_to_route), top_k,
                                   w.data_ptr(), w_scale.data_ptr(), _ptr(bias),
                                   seg_end.data_ptr(), M, N, Kp, E, dt,
                                   None if act is None else ctypes.byref(act), out.data_ptr(),
                                   _ptr(out_scale), ws.data_ptr(), ws.numel(), _stream_of(a)))
    return (out, out_scale) if mx_out else out


def moe_workspace_size_mx(T, H, F, E, K) -> int:
    return load_library().moe_workspace_size_mx(T, H, F, E, K)


def moe_ffn_forward_mx(hidden, hidden_scale, logits, w_gate_up, w_gate_up_scale, w_down,
                       w_down_scale, H: int, F: int, p: RouteParams, act: ActParams,
                       correction_bias=None, expert_ids=None, b_gate_up=None, b_down=None,
                       dtype=torch.bfloat16, out=None, topk_weights_out=None, topk_ids_out=None,
                       ws=None):
    """The routed forward over MX operands: hidden MX e4m3 [T, Hp], weights MX
    e2m1 [E, N1, Hp / 2] and [E, H, Fp / 2]; returns out [T, H] in dtype."""
    lib = load_library()
    _cuda(hidden, hidden_scale, logits, w_gate_up, w_gate_up_scale, w_down, w_down_scale,
          correction_bias, expert_ids, b_gate_up, b_down, out, topk_weights_out, topk_ids_out, ws)
    T, Hp = hidden.shape
    E, N1, half = w_gate_up.shape
    Fp = moe_mx_columns(F)
    if Hp != moe_mx_columns(H) or half * 2 != Hp or N1 != (2 * F if act.kind in _GATED else F) or \
            hidden_scale.shape != (T, Hp // 32) or w_gate_up_scale.shape != (E, N1, Hp // 32) or \
            w_down.shape != (E, H, Fp // 2) or w_down_scale.shape != (E, H, Fp // 32) or \
            logits.shape != (T, E):
        raise ValueError("operands are not MX tensors of matching extents")
    for b, shape in ((b_gate_up, (E, N1)), (b_down, (E, H))):
        if b is not None and (b.dtype != dtype or b.shape != shape):
            raise ValueError("a bias is [E, rows] in the output's dtype")
    if hidden.dtype not in _E4M3 or hidden_scale.dtype not in _E8M0 or \
            w_gate_up.dtype not in _E2M1 or w_gate_up_scale.dtype not in _E8M0 or \
            w_down.dtype not in _E2M1 or w_down_scale.dtype not in _E8M0:
        raise TypeError("hidden is e4m3, the weights e2m1 and the scales e8m0 (or bytes)")
    _typed(correction_bias, torch.float32, "correction_bias")
    _typed(expert_ids, torch.int32, "expert_ids")
    _typed(topk_weights_out, torch.float32, "topk_weights_out")
    _typed(topk_ids_out, torch.int32, "topk_ids_out")
    _fits(correction_bias, (E,), 4, "correction_bias")
    _fits(expert_ids, (T, p.top_k), 4, "expert_ids")
    _fits(topk_weights_out, (T, p.top_k), 4, "topk_weights_out")
    _fits(topk_ids_out, (T, p.top_k), 4, "topk_ids_out")
    if out is None:
        out = torch.empty((T, H), dtype=dtype, device=hidden.device)
    elif out.dtype != dtype or out.shape != (T, H):
        raise ValueError("out is [T, H] in dtype")
    if ws is None:
        ws = _ws(lib.moe_workspace_size_mx(T, H, F, E, p.top_k), hidden.device)
    rp = p if p.dtype == _dt(logits) else _rp(p, logits)
    _check("moe_ffn_forward_mx",
           lib.moe_ffn_forward_mx(hidden.data_ptr(), hidden_scale.data_ptr(), logits.data_ptr(),
                                  w_gate_up.data_ptr(), w_gate_up_scale.data_ptr(),
                                  w_down.data_ptr(), w_down_scale.data_ptr(),
                                  _ptr(correction_bias), _ptr(expert_ids), _ptr(b_gate_up),
                                  _ptr(b_down), T, H, F, E, _dt(out), ctypes.byref(rp),
                                  ctypes.byref(act), out.data_ptr(), _ptr(topk_weights_out),
                                  _ptr(topk_ids_out), ws.data_ptr(), ws.numel(),
                                  _stream_of(hidden)))
    return out


def moe_combine_backward(d_out, expert_out, topk_weights, route_to_row, scale=1.0,
                         d_expert_out=True, d_topk_weights=True):
    """Gradient of moe_combine: (d_expert_out [T * K, H], d_topk_weights [T, K] float32).
    Either is True (made), False or None (left out; expert_out may then be None for the
    weights') or the tensor to write.  topk_weights [T, K]."""
    lib = load_library()
    _together(d_out, expert_out, topk_weights, route_to_row)
    dtype = d_out.dtype
    T, H = d_out.shape
    Tw, K = topk_weights.shape
    M = T * K
    if topk_weights.dtype is not torch.float32 or route_to_row.dtype is not torch.int32 or \
            (expert_out is not None and expert_out.dtype is not dtype):
        raise TypeError("topk_weights is float32, route_to_row int32, expert_out as d_out")
    if Tw != T or K == 0 or route_to_row.numel() != M or \
            (expert_out is not None and expert_out.shape != (M, H)):
        raise ValueError("topk_weights is [T, K], route_to_row [T * K], expert_out [T * K, H]")
    if expert_out is None and not (d_topk_weights is False or d_topk_weights is None):
        raise ValueError("the weights' gradient takes expert_out")
    d_expert_out = _asked(d_expert_out, (M, H), dtype, d_out, "d_expert_out", expert_out)
    d_topk_weights = _asked(d_topk_weights, (T, K), torch.float32, d_out, "d_topk_weights",
                            topk_weights)
    _check("moe_combine_backward",
           lib.moe_combine_backward(d_out.data_ptr(), _ptr(expert_out), topk_weights.data_ptr(),
                                    route_to_row.data_ptr(), T, K, H, _dtype(dtype), scale,
                                    _ptr(d_expert_out), _ptr(d_topk_weights), _stream_of(d_out)))
    return d_expert_out, d_topk_weights


def moe_permute_backward(d_expert_input, route_to_row, K: int, d_hidden=True):
    """Gradient of the permutation: d_hidden [T, H], the sum of a token's K rows of
    d_expert_input [T * K, H]."""
    lib = load_library()
    _together(d_expert_input, route_to_row)
    dtype = d_expert_input.dtype
    M, H = d_expert_input.shape
    if route_to_row.dtype is not torch.int32:
        raise TypeError("route_to_row is int32")
    if K < 1 or M % K or route_to_row.numel() != M:
        raise ValueError("d_expert_input is [T * K, H] and route_to_row [T * K]")
    T = M // K
    d_hidden = _made(d_hidden, (T, H), dtype, d_expert_input, "d_hidden")
    _check("moe_permute_backward",
           lib.moe_permute_backward(d_expert_input.data_ptr(), route_to_row.data_ptr(), T, K, H,
                                    _dtype(dtype), d_hidden.data_ptr(),
                                    _stream_of(d_expert_input)))
    return d_hidden


def moe_act_checkpoint(p, act: ActParams, seg_end=None, out=True, codes=None, scales=None):
    """The activation of a product's rows p [M, N1] and p as MX e4m3 rows: (out [M, F],
    codes [M, N1p], scales [M, N1p / 32]); N1 = 2F for a gated act.  With seg_end, rows
    at and past seg_end[-1] are left alone.  out: True, False, or the tensor to write."""
    lib = load_library()
    _together(p, seg_end, codes, scales)
    dtype = p.dtype
    M, N1 = p.shape
    _segments(seg_end)
    gated = act.kind in _GATED
    if gated and N1 % 2:
        raise ValueError("a gated activation takes pairs of columns")
    F, Np = N1 // 2 if gated else N1, moe_mx_columns(N1)
    out = _asked(out, (M, F), dtype, p, "out")
    if codes is None:
        codes = torch.empty((M, Np), dtype=torch.float8_e4m3fn, device=p.device)
    else:
        _coded(codes, _E4M3, "codes")
        _fits(codes, (M, Np), 1, "codes")
    if scales is None:
        scales = torch.empty((M, Np // 32), dtype=torch.float8_e8m0fnu, device=p.device)
    else:
        _coded(scales, _E8M0, "scales")
        _fits(scales, (M, Np // 32), 1, "scales")
    _check("moe_act_checkpoint",
           lib.moe_act_checkpoint(p.data_ptr(), _ptr(seg_end), M, F,
                                  0 if seg_end is None else seg_end.numel(), _dtype(dtype),
                                  ctypes.byref(act), _ptr(out), codes.data_ptr(),
                                  scales.data_ptr(), _stream_of(p)))
    return out, codes, scales


def moe_act_backward(p, d_out, act: ActParams, scales=None, seg_end=None, d_p=True, out=True):
    """Gradient of the activation: (d_p [M, N1], out [M, F] = act(p) or None) from d_out
    [M, F] and the checkpoint (p its codes, with scales) or p [M, N1] itself.  With
    seg_end, rows at and past seg_end[-1] are left alone."""
    lib = load_library()
    _together(d_out, p, scales, seg_end)
    dtype = d_out.dtype
    M, F = d_out.shape
    N1 = 2 * F if act.kind in _GATED else F
    _segments(seg_end)
    if scales is None:
        _typed(p, dtype, "p")
        if p.shape != (M, N1):
            raise ValueError("p is [M, N1], N1 = 2F for a gated activation")
    else:
        Np = moe_mx_columns(N1)
        _coded(p, _E4M3, "p")
        _coded(scales, _E8M0, "scales")
        if p.shape != (M, Np) or scales.shape != (M, Np // 32):
            raise ValueError("p and scales are [M, N1p] codes and [M, N1p / 32] scales")
    d_p = _made(d_p, (M, N1), dtype, d_out, "d_p")
    out = _asked(out, (M, F), dtype, d_out, "out", d_out)
    _check("moe_act_backward",
           lib.moe_act_backward(p.data_ptr(), _ptr(scales), d_out.data_ptr(), _ptr(seg_end), M, F,
                                0 if seg_end is None else seg_end.numel(), _dtype(dtype),
                                ctypes.byref(act), d_p.data_ptr(), _ptr(out), _stream_of(d_out)))
    return d_p, out


def moe_grouped_gemm_dgrad(d_out, w, seg_end, d_a=True, ws=None):
    """Gradient of a grouped product's rows: d_a [M, K], d_a[m] = d_out[m] . w[e] for the
    rows m of expert e; d_out [M, N], w [E, N, K]."""
    lib = load_library()
    _together(d_out, w, seg_end, ws)
    dtype = d_out.dtype
    M, N = d_out.shape
    E, Nw, K = w.shape
    if w.dtype is not dtype or seg_end.dtype is not torch.int32:
        raise TypeError("w is of d_out's type and seg_end int32")
    if Nw != N or seg_end.numel() != E:
        raise ValueError("d_out is [M, N], w [E, N, K] and seg_end [E]")
    d_a = _made(d_a, (M, K), dtype, d_out, "d_a")
    if ws is None:
        ws = _ws(MOE_STATUS_BYTES, d_out.device)
    _check("moe_grouped_gemm_dgrad",
           lib.moe_grouped_gemm_dgrad(d_out.data_ptr(), w.data_ptr(), seg_end.data_ptr(), M, N, K,
                                      E, _dtype(dtype), d_a.data_ptr(), ws.data_ptr(),
                                      ws.numel() * ws.element_size(), _stream_of(d_out)))
    return d_a


def moe_grouped_gemm_wgrad_workspace_size(M, N, K, E) -> int:
    return load_library().moe_grouped_gemm_wgrad_workspace_size(M, N, K, E)


def moe_grouped_gemm_wgrad(d_out, a, seg_end, bias=False, d_w=True, ws=None):
    """Gradients of a grouped product's weights and bias: (d_w [E, N, K], d_bias [E, N] or
    None), sums over each expert's rows of d_out [M, N] and a [M, K] (zeros for an expert
    without rows).  bias: True, False, or the tensor to write."""
    lib = load_library()
    _together(d_out, a, seg_end, ws)
    dtype = d_out.dtype
    M, N = d_out.shape
    Ma, K = a.shape
    E = seg_end.numel()
    if a.dtype is not dtype or seg_end.dtype is not torch.int32:
        raise TypeError("a is of d_out's type and seg_end int32")
    if Ma != M or E == 0:
        raise ValueError("d_out is [M, N], a [M, K] and seg_end [E]")
    d_w = _made(d_w, (E, N, K), dtype, d_out, "d_w")
    d_bias = _asked(bias, (E, N), dtype, d_out, "bias")
    if ws is None:  # (float32 sums have no parts)
        ws = _ws(MOE_STATUS_BYTES if dtype is torch.float32 else
                 lib.moe_grouped_gemm_wgrad_workspace_size(M, N, K, E), d_out.device)
    _check("moe_grouped_gemm_wgrad",
           lib.moe_grouped_gemm_wgrad(d_out.data_ptr(), a.data_ptr(), seg_end.data_ptr(), M, N, K,
                                      E, _dtype(dtype), d_w.data_ptr(), _ptr(d_bias),
                                      ws.data_ptr(), ws.numel() * ws.element_size(),
                                      _stream_of(d_out)))
    return d_w, d_bias


def moe_route_backward(logits, topk_ids, d_topk_weights, p: RouteParams, d_logits=True):
    """Gradient of moe_route's topk_weights with respect to the logits, [T, E] in the
    logits' type, for the ids that moe_route returned (or was given) under p."""
    lib = load_library()
    _together(logits, topk_ids, d_topk_weights)
    dtype = logits.dtype
    T, E = logits.shape
    if topk_ids.dtype is not torch.int32 or d_topk_weights.dtype is not torch.float32:
        raise TypeError("topk_ids is int32 and d_topk_weights float32")
    if topk_ids.shape != (T, p.top_k) or d_topk_weights.shape != (T, p.top_k):
        raise ValueError("topk_ids and d_topk_weights are [T, K]")
    d_logits = _made(d_logits, (T, E), dtype, logits, "d_logits", logits)
    rp = p if p.dtype == _dtype(dtype) else _rp(p, logits)
    _check("moe_route_backward",
           lib.moe_route_backward(logits.data_ptr(), topk_ids.data_ptr(),
                                  d_topk_weights.data_ptr(), T, E, ctypes.byref(rp),
                                  d_logits.data_ptr(), _stream_of(logits)))
    return d_logits


def moe_shared_expert_workspace_size(T, H, S, dtype=MOE_BF16) -> int:
    return load_library().moe_shared_expert_workspace_size(T, H, S, dtype)


def moe_workspace_size_shared(T, H, F, S, E, K, dtype=MOE_BF16) -> int:
    return load_library().moe_workspace_size_shared(T, H, F, S, E, K, dtype)


def moe_shared_expert_mlp(hidden, w_gate_up, w_down, out=None, ws=None):
    """Shared expert: down(silu(hidden @ gate^T) * (hidden @ up^T)) for every
    token; w_gate_up [2S, H] (gate rows then up rows), w_down [H, S]."""
    lib = load_library()
    _cuda(hidden, w_gate_up, w_down)
    T, H = hidden.shape
    S = w_down.shape[1]
    if out is None:
        out = torch.empty_like(hidden)
    if ws is None:
        ws = _ws(lib.moe_shared_expert_workspace_size(T, H, S, _dt(hidden)), hidden.device)
    _check("moe_shared_expert_mlp",
           lib.moe_shared_expert_mlp(_p(hidden), _p(w_gate_up), _p(w_down), T, H, S, _dt(hidden),
                                     _p(out), _p(ws), ws.numel(), _stream()))
    return out


def moe_ffn_forward_shared(hidden, logits, w_gate_up, w_down, p: RouteParams, act: ActParams,
                           correction_bias=None, shared_w_gate_up=None, shared_w_down=None,
                           routed_out=None, shared_out=None, ws=None):
    """Shared + routed MoE FFN; returns (shared_out or None, routed_out)."""
    lib = load_library()
    _cuda(hidden, logits, w_gate_up, w_down, correction_bias, shared_w_gate_up, shared_w_down)
    T, H = hidden.shape
    E, _, F = w_down.shape
    S = shared_w_down.shape[1] if shared_w_down is not None else 0
    if routed_out is None:
        routed_out = torch.empty_like(hidden)
    if shared_w_gate_up is not None and shared_out is None:
        shared_out = torch.empty_like(hidden)
    if ws is None:
        need = (lib.moe_workspace_size_shared(T, H, F, S, E, p.top_k, _dt(hidden)) if S else
                lib.moe_workspace_size(T, H, F, E, p.top_k, _dt(hidden)))
        ws = _ws(need, hidden.device)
    _check("moe_ffn_forward_shared",
           lib.moe_ffn_forward_shared(_p(hidden), _p(logits), _p(w_gate_up), _p(w_down),
                                      _p(correction_bias), _p(shared_w_gate_up),
                                      _p(shared_w_down), T, H, F, S, E, _dt(hidden),
                                      ctypes.byref(_rp(p, logits)), ctypes.byref(act),
                                      _p(routed_out),
                                      _p(shared_out if shared_w_gate_up is not None else None),
                                      _p(ws), ws.numel(), _stream()))
    return (shared_out if shared_w_gate_up is not None else None), routed_out


def moe_ffn_forward_local(hidden, router_probs, weight_scale, w_gate_up, w_down, K: int,
                          act: ActParams, b_gate_up=None, b_down=None, out=None, ws=None):
    """The expert-parallel rank's layer from its MoERouter outputs
    (router_probs [T, lc], weight_scale [T]) and its lc experts' weights."""
    lib = load_library()
    _cuda(hidden, router_probs, weight_scale, w_gate_up, w_down, b_gate_up, b_down)
    T, H = hidden.shape
    lc, _, F = w_down.shape
    if out is None:
        out = torch.empty_like(hidden)
    if ws is None:
        ws = _ws(lib.moe_workspace_size(T, H, F, lc, min(K, lc), _dt(hidden)), hidden.device)
    _check("moe_ffn_forward_local",
           lib.moe_ffn_forward_local(_p(hidden), _p(router_probs), _p(weight_scale),
                                     _p(w_gate_up), _p(w_down), _p(b_gate_up), _p(b_down), T, H,
                                     F, lc, K, _dt(hidden), _dt(router_probs), ctypes.byref(act),
                                     _p(out), _p(ws),
                                     ws.numel(), _stream()))
    return out


def moe_workspace_size_host(T, H, F, E, K, dtype=MOE_BF16) -> int:
    return load_library().moe_workspace_size_host(T, H, F, E, K, dtype)


def moe_ffn_forward_host(hidden_host, logits_host, w_gate_up, w_down, p: RouteParams,
                         act: ActParams, out_host, ws, correction_bias=None, expert_ids=None,
                         b_gate_up=None, b_down=None, router_probs=None, weight_scale=None):
    """moe_ffn_forward with hidden / logits / out in host memory (pinned for
    asynchronous copies); asynchronous on the current stream.  router_probs /
    weight_scale (device tensors) receive the MoERouter slice outputs when
    ``p`` has a local slice."""
    lib = load_library()
    _cuda(w_gate_up, w_down, correction_bias, expert_ids, b_gate_up, b_down, ws, router_probs,
          weight_scale)
    for t in (hidden_host, logits_host, out_host):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("moe_ffn_forward_host takes contiguous host tensors")
    T, H = hidden_host.shape
    E, _, F = w_down.shape
    _check("moe_ffn_forward_host",
           lib.moe_ffn_forward_host(_p(hidden_host), _p(logits_host), _p(w_gate_up), _p(w_down),
                                    _p(correction_bias), _p(expert_ids), _p(b_gate_up),
                                    _p(b_down), T, H, F, E, _dt(hidden_host),
                                    ctypes.byref(_rp(p, logits_host)),
                                    ctypes.byref(act), _p(out_host), _p(router_probs),
                                    _p(weight_scale), _p(ws), ws.numel(), _stream()))
    return out_host


def moe_clear_status(ws):
    _check("moe_clear_status", load_library().moe_clear_status(_p(ws), _stream()))


def moe_sync_status(ws) -> int:
    """Synchronise the current stream and return (and clear) the status word."""
    return load_library().moe_sync_status(_p(ws), _stream())


def moe_launch_count() -> int:
    return load_library().moe_launch_count()


def moe_set_gemm_simt(enable: bool) -> bool:
    return bool(load_library().moe_set_gemm_simt(int(bool(enable))))


def moe_profile_report() -> dict:
    """Per-stage totals of the forwards recorded since the last report (with
    MOE_PROFILE=1 set before the library loads): {stage: (count, total_us)}."""
    lib = load_library()
    buf = ctypes.create_string_buffer(1 << 16)
    lib.moe_profile_report(buf, len(buf))
    out = {}
    for line in buf.value.decode().splitlines():
        name, count, us = line.split()
        out[name] = (int(count), float(us))
    return out


def moe_test_force_wait_timeout(enable: bool, limit_ns: int = 50_000_000) -> bool:
    """Test hook: make the fused route launch's grid barriers wait for an
    arrival that never comes and give up after ``limit_ns`` (see moe.h)."""
    return bool(load_library().moe_test_force_wait_timeout(int(bool(enable)), int(limit_ns)))


def config_params(cfg):
    """(RouteParams, ActParams) of a synthetic workload recipe (see synth.MoEConfig)."""
    p = route_params(cfg.K, cfg.scoring, cfg.renormalize, cfg.G, cfg.TG, cfg.rsf,
                     cfg.local_start, cfg.local_count, cfg.route_scale)
    a = act_params(cfg.act, cfg.swiglu_fusion, cfg.limit, cfg.alpha, cfg.beta)
    return p, a
