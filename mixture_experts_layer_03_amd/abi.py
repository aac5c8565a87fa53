"""Thin Python binding of libmoe's C ABI (include/moe.h).

Argument marshalling only: every function here takes torch tensors that
already live on the current HIP device, checks nothing beyond what ctypes
needs, passes raw pointers and sizes to the function of the same name in
libmoe.so, and raises MoeError on a non-zero status.  The 8-bit calls
look at their operands' sizes (ValueError): rows of scales are padded, and a
tensor without the padding would be read or written past its end.  The residual
norms and the weighted combine look at shapes, types, strides and devices
(ValueError), since an optional tensor is easily given in another's place.  All arithmetic runs in
the library's kernels.  The library must have been built
(``python -m mixture_experts_layer_03_amd.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

# the in-tree build; MOE_LIBRARY names another build of the same sources
LIB_PATH = os.environ.get("MOE_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK = 0
MOE_F32 = 0
MOE_BF16 = 1
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_ELEMENT = 0, 1, 2, 3

_c_void_p = ctypes.c_void_p
_i32, _i64, _sz = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t

# name -> (restype, argtypes)
_SIGS = {
    "moe_version": (_i32, []),
    "moe_strerror": (ctypes.c_char_p, [_i32]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_router_logits": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i32, _i32,
                                 _c_void_p, _c_void_p]),
    "moe_route": (_i32, [_c_void_p, _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "moe_permute_workspace_size": (_sz, [_i64, _i32, _i32]),
    "moe_permute": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i32, _i32, _i32,
                           _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                           _c_void_p, _sz, _c_void_p]),
    "moe_grouped_ffn_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "moe_grouped_ffn_fwd": (_i32, [_c_void_p, _c_void_p, _i32, _i64, _i32, _i32, _c_void_p,
                                   _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p, _c_void_p,
                                   _c_void_p, _sz, _c_void_p]),
    "moe_grouped_ffn_fwd_noalloc": (_i32, [_c_void_p, _c_void_p, _i32, _i64, _i32, _i32,
                                           _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p,
                                           _c_void_p, _c_void_p, _c_void_p]),
    "moe_grouped_ffn_bwd": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i32,
                                   _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32,
                                   _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                   _c_void_p, _sz, _c_void_p]),
    "moe_combine": (_i32, [_c_void_p, _c_void_p, _i32, _i64, _i32, _i32, _c_void_p, _c_void_p]),
    "moe_combine_bwd": (_i32, [_c_void_p, _c_void_p, _i32, _i64, _i32, _i32, _c_void_p, _c_void_p]),
    "moe_permute_bwd": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i32, _i32, _c_void_p,
                               _c_void_p]),
    "moe_permute_bwd_router": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64,
                                      _i32, _i32, _i32, _c_void_p, _c_void_p]),
    "moe_route_bwd": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32,
                             _c_void_p, _c_void_p, _c_void_p]),
    "moe_router_logits_bwd_workspace_size": (_sz, [_i64, _i32, _i32]),
    "moe_router_logits_bwd": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _i64, _i32, _i32,
                                     _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "moe_route_biased": (_i32, [_c_void_p, _c_void_p, _i64, _i32, _i32, _c_void_p, _c_void_p,
                                _c_void_p]),
    "moe_expert_load_workspace_size": (_sz, [_i64, _i32, _i32]),
    "moe_expert_load": (_i32, [_c_void_p, _i64, _i64, _i32, _i32, _c_void_p, _c_void_p, _sz,
                               _c_void_p]),
    "moe_bias_update": (_i32, [_c_void_p, _i64, _i32, _i32, ctypes.c_float, _c_void_p,
                               _c_void_p]),
    "moe_aux_loss_workspace_size": (_sz, [_i64, _i32]),
    "moe_aux_loss": (_i32, [_c_void_p, _c_void_p, _i64, _i64, _i32, _i32, ctypes.c_float,
                            _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "moe_grouped_ffn_lora_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "moe_grouped_ffn_fwd_lora": (_i32, [_c_void_p, _c_void_p, _i32, _i64, _i32, _i32, _c_void_p,
                                        _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                        _c_void_p, _i32, ctypes.c_float, _i32, _c_void_p,
                                        _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                        _sz, _c_void_p]),
    "moe_grouped_ffn_bwd_lora": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32, _i64,
                                        _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                        _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32,
                                        ctypes.c_float, _c_void_p, _c_void_p, _i32, _c_void_p,
                                        _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                        _c_void_p, _c_void_p, _sz, _c_void_p]),
    "moe_grouped_ffn_lora_bwd_saved": (_i32, [_c_void_p, _sz, _i64, _i32, _i32, _i32, _i32,
                                              ctypes.POINTER(_c_void_p), ctypes.POINTER(_c_void_p),
                                              ctypes.POINTER(_c_void_p)]),
    "moe_grouped_ffn_fwd_gather": (_i32, [_c_void_p, _i64, _c_void_p, _i32, _c_void_p, _i32,
                                          _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                          _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "moe_grouped_ffn_bwd_gather": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p,
                                          _c_void_p, _i32, _c_void_p,
                                          _c_void_p, _c_void_p, _i32, _i32, _i32, _c_void_p,
                                          _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                          _c_void_p, _c_void_p, _c_void_p, _sz, _c_void_p]),
    "moe_route_scored": (_i32, [_c_void_p, _c_void_p, _i64, _i32, _i32, _i32, _i32, _i32, _i32,
                                _i32, ctypes.c_float, _c_void_p, _c_void_p, _c_void_p]),
    "moe_route_scored_bwd": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i64,
                                    _i32, _i32, _i32, _i32, ctypes.c_float, _c_void_p, _c_void_p,
                                    _c_void_p]),
    "moe_fp8_scale_cols": (_i32, [_i32]),
    "moe_quant_rows_fp8": (_i32, [_c_void_p, _i32, _i64, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "moe_quant_weights_fp8": (_i32, [_c_void_p, _i32, _i32, _i32, _i32, _c_void_p, _c_void_p,
                                     _c_void_p, _c_void_p, _c_void_p]),
    "moe_grouped_gemm_fp8": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p, _i32, _i64,
                                    _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p]),
    "moe_grouped_ffn_fwd_fp8": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p, _i32,
                                       _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p,
                                       _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                       _c_void_p]),
    "moe_residual_norm": (_i32, [_c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p,
                                 ctypes.c_float, ctypes.c_float, _i32, _i64, _i32, _c_void_p,
                                 _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "moe_residual_norm_bwd_workspace_size": (_sz, [_i64, _i32]),
    "moe_residual_norm_bwd": (_i32, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _i32,
                                     _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_float,
                                     _i32, _i64, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                     _c_void_p, _c_void_p, _sz, _c_void_p]),
    "moe_combine_weighted": (_i32, [_c_void_p, _i64, _c_void_p, _c_void_p, _i32, _i64, _i32, _i32,
                                    _c_void_p, _c_void_p]),
    "moe_combine_weighted_bwd": (_i32, [_c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p, _i32,
                                        _i64, _i32, _i32, _c_void_p, _c_void_p, _c_void_p]),
    "moe_combine_residual_norm": (_i32, [_c_void_p, _i64, _c_void_p, _c_void_p, _i32, _c_void_p,
                                         _c_void_p, _i32, _c_void_p, _c_void_p, ctypes.c_float,
                                         ctypes.c_float, _i32, _i64, _i32, _c_void_p, _c_void_p,
                                         _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "moe_adamw_step": (_i32, [_c_void_p, _i32, _i32, _i32, _i32, ctypes.c_double, ctypes.c_double,
                              ctypes.c_double, ctypes.c_double, _i64, ctypes.c_uint64, _c_void_p,
                              _c_void_p, _c_void_p, _c_void_p]),
    "moe_timing_enable": (_i32, [_i32]),
    "moe_timing_reset": (_i32, []),
    "moe_timing_query": (_i32, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_double),
                                ctypes.POINTER(ctypes.c_int64)]),
}

_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__("%s failed (status %d): %s" % (fn, status, msg))
        self.status = status


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe.so is not built (%s); run "
                               "`python -m mixture_experts_layer_03_amd.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _p(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


_current_stream = None


def _stream(stream) -> Optional[int]:
    """The given stream, or the current stream of the current device (taken
    without building a Stream object where torch offers that: 0.4 against 2.6
    us, as much as a small kernel's launch)."""
    if stream is not None:
        return stream
    global _current_stream
    if _current_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            _current_stream = lambda: torch.cuda.current_stream().cuda_stream
        else:
            _current_stream = lambda: raw(torch.cuda.current_device())
    return _current_stream()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float32:
        return MOE_F32
    raise TypeError("unsupported dtype %s" % t.dtype)


def _check(fn: str, rc: int):
    if rc != MOE_OK:
        raise MoeError(fn, rc, (lib().moe_last_error() or b"").decode())


# ---------------------------------------------------------------- entry points

def moe_router_logits(x, w_r, bias, logit_add, logits, stream=None):
    T, d = x.shape
    E = w_r.shape[0]
    _check("moe_router_logits", lib().moe_router_logits(
        _p(x), _p(w_r), _p(bias), _p(logit_add), _dtype_code(x), T, d, E, _p(logits),
        _stream(stream)))


def moe_route(logits, k, topk_idx, topk_w, stream=None):
    T, E = logits.shape
    _check("moe_route", lib().moe_route(_p(logits), T, E, k, _p(topk_idx), _p(topk_w),
                                        _stream(stream)))


def moe_permute_workspace_size(T, E, k) -> int:
    return int(lib().moe_permute_workspace_size(T, E, k))


def moe_permute(x, topk_idx, topk_w, T, d, E, k, counts, offsets, slot_to_row, row_to_slot,
                x_perm, w_perm, ws, dtype=None, stream=None):
    dt = _dtype_code(x) if x is not None else (MOE_BF16 if dtype is None else dtype)
    _check("moe_permute", lib().moe_permute(
        _p(x), _p(topk_idx), _p(topk_w), dt, T, d, E, k, _p(counts), _p(offsets),
        _p(slot_to_row), _p(row_to_slot), _p(x_perm), _p(w_perm), _p(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_grouped_ffn_workspace_size(R, E, d, f, dtype) -> int:
    return int(lib().moe_grouped_ffn_workspace_size(R, E, d, f, dtype))


def moe_grouped_ffn_fwd(x_perm, offsets, E, w_gu, w_down, row_scale, gu, h, y_perm, ws,
                        stream=None):
    R, d = x_perm.shape
    f = w_down.shape[2]
    _check("moe_grouped_ffn_fwd", lib().moe_grouped_ffn_fwd(
        _p(x_perm), _p(offsets), E, R, d, f, _p(w_gu), _p(w_down), _p(row_scale),
        _dtype_code(x_perm), _p(gu), _p(h), _p(y_perm), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_grouped_ffn_fwd_noalloc(x_perm, offsets, E, w_gu, w_down, row_scale, gu, h, y_perm,
                                stream=None):
    R, d = x_perm.shape
    f = w_down.shape[2]
    _check("moe_grouped_ffn_fwd_noalloc", lib().moe_grouped_ffn_fwd_noalloc(
        _p(x_perm), _p(offsets), E, R, d, f, _p(w_gu), _p(w_down), _p(row_scale),
        _dtype_code(x_perm), _p(gu), _p(h), _p(y_perm), _stream(stream)))


def moe_grouped_ffn_bwd(x_perm, gu, h, offsets, E, w_gu, w_down, row_scale, dy_perm, dgu,
                        dx_perm, dw_gu, dw_down, d_row_scale, ws, stream=None):
    R, d = x_perm.shape
    f = w_down.shape[2]
    _check("moe_grouped_ffn_bwd", lib().moe_grouped_ffn_bwd(
        _p(x_perm), _p(gu), _p(h), _p(offsets), E, R, d, f, _p(w_gu), _p(w_down),
        _p(row_scale), _p(dy_perm), _dtype_code(w_gu), _p(dgu), _p(dx_perm), _p(dw_gu),
        _p(dw_down), _p(d_row_scale), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_grouped_ffn_fwd_gather(x, row_to_slot, k, offsets, E, w_gu, w_down, row_scale, gu, h,
                               y_perm, ws, stream=None):
    T, d = x.shape
    f = w_down.shape[2]
    _check("moe_grouped_ffn_fwd_gather", lib().moe_grouped_ffn_fwd_gather(
        _p(x), T, _p(row_to_slot), k, _p(offsets), E, d, f, _p(w_gu), _p(w_down), _p(row_scale),
        _p(gu), _p(h), _p(y_perm), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_grouped_ffn_bwd_gather(x, dy, row_to_slot, slot_to_row, k, gu, h, offsets, E, w_gu,
                               w_down, row_scale, dgu, dx_perm, dw_gu, dw_down, d_row_scale, ws,
                               stream=None, x_perm=None):
    """x_perm given: the dW_gu GEMM reads it instead of gathering x."""
    T, d = dy.shape
    f = w_down.shape[2]
    _check("moe_grouped_ffn_bwd_gather", lib().moe_grouped_ffn_bwd_gather(
        _p(x), _p(x_perm), _p(dy), T, _p(row_to_slot), _p(slot_to_row), k, _p(gu), _p(h),
        _p(offsets), E, d, f,
        _p(w_gu), _p(w_down), _p(row_scale), _p(dgu), _p(dx_perm), _p(dw_gu), _p(dw_down),
        _p(d_row_scale), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_combine(y_perm, slot_to_row, T, k, y, stream=None):
    d = y_perm.shape[1]
    _check("moe_combine", lib().moe_combine(_p(y_perm), _p(slot_to_row), _dtype_code(y_perm),
                                            T, d, k, _p(y), _stream(stream)))


def moe_combine_bwd(dy, slot_to_row, k, dy_perm, stream=None):
    T, d = dy.shape
    _check("moe_combine_bwd", lib().moe_combine_bwd(_p(dy), _p(slot_to_row), _dtype_code(dy),
                                                    T, d, k, _p(dy_perm), _stream(stream)))


def moe_permute_bwd(dx_perm, slot_to_row, dx_add, T, k, dx, stream=None):
    d = dx_perm.shape[1]
    _check("moe_permute_bwd", lib().moe_permute_bwd(_p(dx_perm), _p(slot_to_row), _p(dx_add),
                                                    _dtype_code(dx_perm), T, d, k, _p(dx),
                                                    _stream(stream)))


def moe_permute_bwd_router(dx_perm, slot_to_row, d_logits, w_r, T, k, dx, stream=None):
    d = dx_perm.shape[1]
    E = w_r.shape[0]
    _check("moe_permute_bwd_router", lib().moe_permute_bwd_router(
        _p(dx_perm), _p(slot_to_row), _p(d_logits), _p(w_r), _dtype_code(dx_perm), T, d, E, k,
        _p(dx), _stream(stream)))


def moe_route_bwd(topk_idx, topk_w, d_row_scale, slot_to_row, E, d_topk_w, d_logits,
                  stream=None):
    T, k = topk_idx.shape
    _check("moe_route_bwd", lib().moe_route_bwd(_p(topk_idx), _p(topk_w), _p(d_row_scale),
                                                _p(slot_to_row), T, E, k, _p(d_topk_w),
                                                _p(d_logits), _stream(stream)))


def moe_router_logits_bwd_workspace_size(T, d, E) -> int:
    return int(lib().moe_router_logits_bwd_workspace_size(T, d, E))


def moe_router_logits_bwd(x, w_r, d_logits, dx_router, dw_r, ws, stream=None):
    T, d = x.shape
    E = w_r.shape[0]
    _check("moe_router_logits_bwd", lib().moe_router_logits_bwd(
        _p(x), _p(w_r), _p(d_logits), _dtype_code(x), T, d, E, _p(dx_router), _p(dw_r), _p(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_route_biased(logits, sel_bias, k, topk_idx, topk_w, stream=None):
    T, E = logits.shape
    _check("moe_route_biased", lib().moe_route_biased(_p(logits), _p(sel_bias), T, E, k,
                                                      _p(topk_idx), _p(topk_w), _stream(stream)))


def moe_expert_load_workspace_size(T, E, k) -> int:
    return int(lib().moe_expert_load_workspace_size(T, E, k))


def moe_expert_load(topk_idx, n_valid, E, load, ws, stream=None):
    T, k = topk_idx.shape
    _check("moe_expert_load", lib().moe_expert_load(
        _p(topk_idx), T, n_valid, E, k, _p(load), _p(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_bias_update(load, n_valid, k, rate, sel_bias, stream=None):
    E = load.shape[0]
    _check("moe_bias_update", lib().moe_bias_update(_p(load), n_valid, E, k, float(rate),
                                                    _p(sel_bias), _stream(stream)))


def moe_aux_loss_workspace_size(T, E) -> int:
    return int(lib().moe_aux_loss_workspace_size(T, E))


def moe_aux_loss(logits, load, n_valid, k, coeff, aux_out, d_logits, ws, stream=None):
    T, E = logits.shape
    _check("moe_aux_loss", lib().moe_aux_loss(
        _p(logits), _p(load), T, n_valid, E, k, float(coeff), _p(aux_out), _p(d_logits), _p(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))


def moe_grouped_ffn_lora_workspace_size(R, E, d, f, r) -> int:
    return int(lib().moe_grouped_ffn_lora_workspace_size(R, E, d, f, r))


def moe_grouped_ffn_fwd_lora(x_perm, offsets, E, w_gu, w_down, row_scale, a_gu, b_gu, a_dn, b_dn,
                             scale, z_gu, z_dn, gu, h, y_perm, ws, stream=None):
    R, d = x_perm.shape
    f = w_down.shape[2]
    r = a_gu.shape[1]
    _check("moe_grouped_ffn_fwd_lora", lib().moe_grouped_ffn_fwd_lora(
        _p(x_perm), _p(offsets), E, R, d, f, _p(w_gu), _p(w_down), _p(row_scale), _p(a_gu),
        _p(b_gu), _p(a_dn), _p(b_dn), r, float(scale), _dtype_code(x_perm), _p(z_gu), _p(z_dn),
        _p(gu), _p(h), _p(y_perm), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_grouped_ffn_bwd_lora(x_perm, gu, h, offsets, E, w_gu, w_down, row_scale, dy_perm, a_gu,
                             b_gu, a_dn, b_dn, scale, z_gu, z_dn, dgu, dx_perm, d_row_scale,
                             da_gu, db_gu, da_dn, db_dn, ws, stream=None):
    R, d = x_perm.shape
    f = w_down.shape[2]
    r = a_gu.shape[1]
    _check("moe_grouped_ffn_bwd_lora", lib().moe_grouped_ffn_bwd_lora(
        _p(x_perm), _p(gu), _p(h), _p(offsets), E, R, d, f, _p(w_gu), _p(w_down), _p(row_scale),
        _p(dy_perm), _p(a_gu), _p(b_gu), _p(a_dn), _p(b_dn), r, float(scale), _p(z_gu), _p(z_dn),
        _dtype_code(w_gu), _p(dgu), _p(dx_perm), _p(d_row_scale), _p(da_gu), _p(db_gu),
        _p(da_dn), _p(db_dn), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_grouped_ffn_lora_bwd_saved(ws, R, E, d, f, r):
    """Views [R, r] (bf16) of u_dn, store(w u_dn) and u_gu inside the LoRA
    backward's workspace ws (a uint8 device tensor)."""
    import torch
    ptrs = [_c_void_p(), _c_void_p(), _c_void_p()]
    nbytes = ws.numel() * ws.element_size()
    _check("moe_grouped_ffn_lora_bwd_saved", lib().moe_grouped_ffn_lora_bwd_saved(
        _p(ws), nbytes, R, E, d, f, r, ctypes.byref(ptrs[0]), ctypes.byref(ptrs[1]),
        ctypes.byref(ptrs[2])))
    base = ws.data_ptr()
    out = []
    for p in ptrs:
        off = int(p.value) - base
        out.append(ws[off:off + 2 * R * r].view(torch.bfloat16).view(R, r))
    return tuple(out)


def moe_route_scored(logits, sel_bias, k, topk_idx, topk_w, score=MOE_SCORE_SOFTMAX, n_group=1,
                     topk_group=1, group_top=1, renorm=True, scale=1.0, stream=None):
    """sel_bias: [E] or None."""
    T, E = logits.shape
    _check("moe_route_scored", lib().moe_route_scored(
        _p(logits), _p(sel_bias), T, E, k, score, n_group, topk_group, group_top,
        1 if renorm else 0, float(scale), _p(topk_idx), _p(topk_w), _stream(stream)))


def moe_route_scored_bwd(logits, topk_idx, topk_w, d_row_scale, slot_to_row, d_topk_w, d_logits,
                         score=MOE_SCORE_SOFTMAX, renorm=True, scale=1.0, stream=None):
    """slot_to_row None: d_row_scale is in slot order; d_topk_w may be None."""
    T, E = logits.shape
    k = topk_idx.shape[1]
    _check("moe_route_scored_bwd", lib().moe_route_scored_bwd(
        _p(logits), _p(topk_idx), _p(topk_w), _p(d_row_scale), _p(slot_to_row), T, E, k, score,
        1 if renorm else 0, float(scale), _p(d_topk_w), _p(d_logits), _stream(stream)))


def moe_fp8_scale_cols(K) -> int:
    return int(lib().moe_fp8_scale_cols(K))


def _pitch(t, cols):
    """Whether the rows of a scale tensor are not `cols` long (a flat one has none)."""
    return t.shape[-1] != cols and t.dim() > 1


def _misfit(fn, *operands):
    """Raises for the first (name, tensor, rows, cols, bytes per element) that
    does not hold its rows; cols is given for scale tensors, whose rows are
    padded to moe_fp8_scale_cols, and else counted into rows."""
    for name, t, rows, cols, size in operands:
        if t is None:
            continue
        need = rows * (cols or 1) * size
        if (cols and _pitch(t, cols)) or t.nbytes < need or not t.is_contiguous():
            raise ValueError("%s: %s must be contiguous and hold %d bytes%s, not %s of %s"
                             % (fn, name, need, " in rows of %d" % cols if cols else "",
                                tuple(t.shape), t.dtype))


def moe_quant_rows_fp8(x, q, scale, stream=None):
    R, K = x.shape
    cols = -(-K // 512) * 4
    if (q.nbytes < R * K or _pitch(scale, cols) or scale.nbytes < R * cols
            or not (x.is_contiguous() and q.is_contiguous() and scale.is_contiguous())):
        _misfit("moe_quant_rows_fp8", ("x", x, 0, 0, 1), ("q", q, R * K, 0, 1),
                ("scale", scale, R, cols, 1))
    _check("moe_quant_rows_fp8", lib().moe_quant_rows_fp8(
        _p(x), _dtype_code(x), R, K, _p(q), _p(scale), _stream(stream)))


def moe_quant_weights_fp8(w, q, scale, qt=None, scale_t=None, stream=None):
    E, N, K = w.shape
    _misfit("moe_quant_weights_fp8", ("w", w, 0, 0, 1), ("q", q, E * N * K, 0, 1),
            ("scale", scale, E * -(-N // 128), -(-K // 512) * 4, 1), ("qt", qt, E * N * K, 0, 1),
            ("scale_t", scale_t, E * -(-K // 128), -(-N // 512) * 4, 1))
    _check("moe_quant_weights_fp8", lib().moe_quant_weights_fp8(
        _p(w), _dtype_code(w), E, N, K, _p(q), _p(scale), _p(qt), _p(scale_t), _stream(stream)))


def moe_grouped_gemm_fp8(a, a_scale, offsets, b, b_scale, row_scale, c, row_to_slot=None, k=1,
                         stream=None):
    """With row_to_slot, a holds token rows and row r reads token row_to_slot[r] / k."""
    R = c.shape[0]
    E, N, K = b.shape
    rows, cols, blocks = R if row_to_slot is None else R // max(k, 1), -(-K // 512) * 4, -(-N // 128)
    if (a.nbytes < rows * K or a_scale.nbytes < rows * cols or _pitch(a_scale, cols)
            or b_scale.nbytes < E * blocks * cols or _pitch(b_scale, cols)
            or offsets.nbytes < 4 * E + 4 or c.nbytes < 2 * R * N
            or (row_to_slot is not None and row_to_slot.nbytes < 4 * R)
            or (row_scale is not None and row_scale.nbytes < 4 * R)
            or not (a.is_contiguous() and a_scale.is_contiguous() and b.is_contiguous()
                    and b_scale.is_contiguous() and c.is_contiguous())):
        _misfit("moe_grouped_gemm_fp8", ("a", a, rows * K, 0, 1), ("a_scale", a_scale, rows, cols, 1),
                ("offsets", offsets, E + 1, 0, 4), ("b", b, 0, 0, 1),
                ("b_scale", b_scale, E * blocks, cols, 1), ("row_scale", row_scale, R, 0, 4),
                ("c", c, R * N, 0, 2), ("row_to_slot", row_to_slot, R, 0, 4))
    _check("moe_grouped_gemm_fp8", lib().moe_grouped_gemm_fp8(
        _p(a), _p(a_scale), _p(row_to_slot), k, _p(offsets), E, R, N, K, _p(b), _p(b_scale),
        _p(row_scale), _p(c), _stream(stream)))


def moe_grouped_ffn_fwd_fp8(x, x_scale, offsets, w_gu, w_gu_scale, w_down, w_down_scale,
                            row_scale, h, h_scale, y_perm, row_to_slot=None, k=1, stream=None):
    """With row_to_slot, x holds token rows and row r reads token row_to_slot[r] / k."""
    R, d = y_perm.shape
    E, _, f = w_down.shape
    rows = R if row_to_slot is None else R // max(k, 1)
    cols, cols_f = -(-d // 512) * 4, -(-f // 512) * 4
    gu_blocks, blocks = -(-2 * f // 128), -(-d // 128)
    if (x.nbytes < rows * d or x_scale.nbytes < rows * cols or _pitch(x_scale, cols)
            or w_gu.nbytes < 2 * E * f * d or w_down.nbytes < E * d * f
            or w_gu_scale.nbytes < E * gu_blocks * cols or _pitch(w_gu_scale, cols)
            or w_down_scale.nbytes < E * blocks * cols_f or _pitch(w_down_scale, cols_f)
            or h.nbytes < R * f or h_scale.nbytes < R * cols_f or _pitch(h_scale, cols_f)
            or offsets.nbytes < 4 * E + 4 or y_perm.nbytes < 2 * R * d
            or (row_to_slot is not None and row_to_slot.nbytes < 4 * R)
            or (row_scale is not None and row_scale.nbytes < 4 * R)
            or not (x.is_contiguous() and x_scale.is_contiguous() and w_gu.is_contiguous()
                    and w_gu_scale.is_contiguous() and w_down.is_contiguous()
                    and w_down_scale.is_contiguous() and h.is_contiguous()
                    and h_scale.is_contiguous() and y_perm.is_contiguous())):
        _misfit("moe_grouped_ffn_fwd_fp8", ("x", x, rows * d, 0, 1),
                ("x_scale", x_scale, rows, cols, 1), ("offsets", offsets, E + 1, 0, 4),
                ("w_gu", w_gu, 2 * E * f * d, 0, 1),
                ("w_gu_scale", w_gu_scale, E * gu_blocks, cols, 1),
                ("w_down", w_down, E * d * f, 0, 1),
                ("w_down_scale", w_down_scale, E * blocks, cols_f, 1),
                ("row_scale", row_scale, R, 0, 4), ("h", h, R * f, 0, 1),
                ("h_scale", h_scale, R, cols_f, 1), ("y_perm", y_perm, R * d, 0, 2),
                ("row_to_slot", row_to_slot, R, 0, 4))
    _check("moe_grouped_ffn_fwd_fp8", lib().moe_grouped_ffn_fwd_fp8(
        _p(x), _p(x_scale), _p(row_to_slot), k, _p(offsets), E, R, d, f, _p(w_gu),
        _p(w_gu_scale), _p(w_down), _p(w_down_scale), _p(row_scale), _p(h), _p(h_scale),
        _p(y_perm), _stream(stream)))


_torch = None


def _types():
    """(torch, torch.float32, index of the current device); torch is imported by the first call."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch, _torch.float32, _torch._C._cuda_getDevice() if _torch.cuda.is_initialized() else 0


def _fits(fn, here, *groups):
    """Raises for the first tensor that is not a contiguous one of its group's shape and type on the
    current device; groups: (names, tensors, shape, type), None passes."""
    for names, tensors, shape, dtype in groups:
        for t in tensors:
            if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()
                                  or t.get_device() != here):
                name = names.split()[[x is t for x in tensors].index(True)]
                raise ValueError("%s: %s must be a contiguous %s of %s on the current device, not %s of %s%s on %s"
                                 % (fn, name, tuple(shape), dtype, tuple(t.shape), t.dtype,
                                    "" if t.is_contiguous() else " with strides", t.device))


def _gate_kind(fn, gate, T, d, dtype, f32):
    """(kind, shape, type) of a gate by its shape: [d] a channel's, [T,1] a token's (fp32), [T,d]."""
    if gate is None:
        return MOE_GATE_NONE, None, None
    if gate.shape == (d,):
        return MOE_GATE_CHANNEL, (d,), dtype
    if gate.shape == (T, 1):
        return MOE_GATE_TOKEN, (T, 1), f32
    if gate.shape == (T, d):
        return MOE_GATE_ELEMENT, (T, d), dtype
    raise ValueError("%s: gate must be [d], [T,1] or [T,d], not %s" % (fn, tuple(gate.shape)))


def moe_residual_norm(x, y, out, n, w_post=None, w_pre=None, gate=None, res_scale=1.0, eps=1e-6,
                      rstd_post=None, rstd_pre=None, stream=None):
    """y None: n alone, the norm of x.  gate: [d], [T,1] (fp32) or [T,d]."""
    _, f32, here = _types()
    fn, some = "moe_residual_norm", x if y is None else y
    dt = some.dtype
    T, d = some.shape
    kind, gshape, gtype = _gate_kind(fn, gate, T, d, dt, f32)
    _fits(fn, here, ("x y out n", (x, y, out, n), (T, d), dt), ("w_post w_pre", (w_post, w_pre), (d,), dt),
          ("rstd_post rstd_pre", (rstd_post, rstd_pre), (T,), f32), ("gate", (gate,), gshape, gtype))
    _check(fn, lib().moe_residual_norm(
        _p(x), _p(y), _p(gate), kind, _p(w_post), _p(w_pre), res_scale, eps, _dtype_code(some), T, d,
        _p(out), _p(n), _p(rstd_post), _p(rstd_pre), _stream(stream)))


def moe_residual_norm_bwd_workspace_size(T, d) -> int:
    return int(lib().moe_residual_norm_bwd_workspace_size(T, d))


def moe_residual_norm_bwd(d_out, d_n, out, y, d_x, d_y, ws, w_post=None, w_pre=None, gate=None,
                          res_scale=1.0, rstd_post=None, rstd_pre=None, d_w_post=None,
                          d_w_pre=None, d_gate=None, stream=None):
    _, f32, here = _types()
    fn, some = "moe_residual_norm_bwd", d_n if d_out is None else d_out
    dt = some.dtype
    T, d = some.shape
    kind, gshape, gtype = _gate_kind(fn, gate, T, d, dt, f32)
    _fits(fn, here, ("d_out d_n out y d_x d_y", (d_out, d_n, out, y, d_x, d_y), (T, d), dt),
          ("w_post w_pre", (w_post, w_pre), (d,), dt), ("gate", (gate,), gshape, gtype),
          ("rstd_post rstd_pre", (rstd_post, rstd_pre), (T,), f32),
          ("d_w_post d_w_pre", (d_w_post, d_w_pre), (d,), f32),
          ("d_gate", (d_gate,), gshape, f32 if kind == MOE_GATE_CHANNEL else gtype))
    if ws is not None and (ws.get_device() != here or not ws.is_contiguous()):
        raise ValueError("%s: ws must be contiguous and on the current device, not %s%s on %s"
                         % (fn, tuple(ws.shape), "" if ws.is_contiguous() else " with strides", ws.device))
    _check(fn, lib().moe_residual_norm_bwd(
        _p(d_out), _p(d_n), _p(out), _p(y), _p(gate), kind, _p(w_post), _p(w_pre), _p(rstd_post),
        _p(rstd_pre), res_scale, _dtype_code(some), T, d, _p(d_x), _p(d_y), _p(d_w_post),
        _p(d_w_pre), _p(d_gate), _p(ws), 0 if ws is None else ws.nbytes, _stream(stream)))


def moe_combine_weighted(y_perm, slot_to_row, weights, y, stream=None):
    torch, f32, here = _types()
    fn, dt = "moe_combine_weighted", y.dtype
    T, k = weights.shape
    d = y.shape[1]
    _fits(fn, here, ("y_perm", (y_perm,), (y_perm.shape[0], d), dt), ("y", (y,), (T, d), dt),
          ("slot_to_row", (slot_to_row,), (T * k,), torch.int32), ("weights", (weights,), (T, k), f32))
    _check(fn, lib().moe_combine_weighted(_p(y_perm), y_perm.shape[0], _p(slot_to_row), _p(weights),
                                          _dtype_code(y), T, d, k, _p(y), _stream(stream)))


def moe_combine_weighted_bwd(dy, y_perm, slot_to_row, weights, dy_perm, d_row_scale, stream=None):
    torch, f32, here = _types()
    fn, dt = "moe_combine_weighted_bwd", dy.dtype
    T, k = weights.shape
    d = dy.shape[1]
    R = dy_perm.shape[0] if y_perm is None else y_perm.shape[0]
    _fits(fn, here, ("dy", (dy,), (T, d), dt), ("y_perm dy_perm", (y_perm, dy_perm), (R, d), dt),
          ("slot_to_row", (slot_to_row,), (T * k,), torch.int32), ("weights", (weights,), (T, k), f32),
          ("d_row_scale", (d_row_scale,), (R,), f32))
    _check(fn, lib().moe_combine_weighted_bwd(
        _p(dy), _p(y_perm), R, _p(slot_to_row), _p(weights), _dtype_code(dy), T, d, k, _p(dy_perm),
        _p(d_row_scale), _stream(stream)))


def moe_combine_residual_norm(y_perm, slot_to_row, weights, k, x, out, n, y=None, w_post=None,
                              w_pre=None, gate=None, res_scale=1.0, eps=1e-6, rstd_post=None,
                              rstd_pre=None, stream=None):
    """weights None: the rows carry them already.  y: the combined rows, stored for a backward."""
    torch, f32, here = _types()
    fn, dt = "moe_combine_residual_norm", out.dtype
    T, d = out.shape
    kind, gshape, gtype = _gate_kind(fn, gate, T, d, dt, f32)
    _fits(fn, here, ("x y out n", (x, y, out, n), (T, d), dt), ("y_perm", (y_perm,), (y_perm.shape[0], d), dt),
          ("slot_to_row", (slot_to_row,), (T * k,), torch.int32), ("weights", (weights,), (T, k), f32),
          ("w_post w_pre", (w_post, w_pre), (d,), dt), ("rstd_post rstd_pre", (rstd_post, rstd_pre), (T,), f32),
          ("gate", (gate,), gshape, gtype))
    _check(fn, lib().moe_combine_residual_norm(
        _p(y_perm), y_perm.shape[0], _p(slot_to_row), _p(weights), k, _p(x), _p(gate), kind, _p(w_post), _p(w_pre),
        res_scale, eps, _dtype_code(out), T, d, _p(y), _p(out), _p(n), _p(rstd_post), _p(rstd_pre),
        _stream(stream)))


class AdamwTensor(ctypes.Structure):
    """moe_adamw_tensor"""
    _fields_ = [("param", _c_void_p), ("grad", _c_void_p), ("master", _c_void_p), ("m", _c_void_p),
                ("v", _c_void_p), ("m_scale", _c_void_p), ("v_scale", _c_void_p), ("numel", _i64),
                ("weight_decay", ctypes.c_double)]


def moe_adamw_step(tensors, n, param_dtype, grad_dtype, state_bits, lr, beta1, beta2, eps, step,
                   seed, grad_scale=None, lr_dev=None, step_dev=None, stream=None):
    """tensors: a ctypes array of n AdamwTensor."""
    _check("moe_adamw_step", lib().moe_adamw_step(
        ctypes.addressof(tensors), n, param_dtype, grad_dtype, state_bits, lr, beta1, beta2, eps,
        step, seed, _p(grad_scale), _p(lr_dev), _p(step_dev), _stream(stream)))


def moe_timing_enable(on: bool):
    _check("moe_timing_enable", lib().moe_timing_enable(1 if on else 0))


def moe_timing_reset():
    _check("moe_timing_reset", lib().moe_timing_reset())


def moe_timing_query(name: Optional[str]):
    ms = ctypes.c_double(0.0)
    n = ctypes.c_int64(0)
    _check("moe_timing_query", lib().moe_timing_query(None if name is None else name.encode(),
                                                      ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value
