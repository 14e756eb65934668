"""Thin Python binding of libmoe's C ABI (include/moe.h).

Argument marshalling only: every function takes torch tensors (device memory
owned by the caller), passes their data pointers, the current CUDA stream and the
shape struct to the C entry point of the same name, and raises MoeError on a
non-zero status.  Every step of the layer runs in libmoe's kernels; if the
library is missing this module raises at import time instead of falling back to
anything else.
"""
from __future__ import annotations

import ctypes
import os
from bisect import bisect_left

import torch

from .synth import Workload

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, 1, 2, 3
MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_DEVICE_CHECK = 4, 5, 6
MOE_F32, MOE_BF16, MOE_MXFP8 = 0, 1, 2
DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "mxfp8": MOE_MXFP8}

ENTRY_POINTS = (
    "moe_workspace_bytes", "moe_workspace_init", "moe_last_device_status", "moe_status_string",
    "moe_quantize_mxfp8", "moe_quantize_nvfp4", "moe_macro_workspace_bytes", "moe_forward_macrobatched",
    "moe_route_topk", "moe_layout", "moe_dispatch_pull", "moe_expert_ffn",
    "moe_combine", "moe_forward", "moe_forward_fused", "moe_min_minibatch", "moe_layout_noalloc",
    "moe_pack_expert_weights", "moe_backward_workspace_bytes", "moe_pack_expert_weights_dgrad",
    "moe_expert_ffn_train", "moe_forward_train", "moe_reverse_combine", "moe_expert_ffn_dgrad",
    "moe_reverse_dispatch", "moe_router_wgrad", "moe_backward", "moe_expert_wgrad",
    "moe_embedding", "moe_embedding_workspace_bytes", "moe_embedding_backward", "moe_token_logprobs",
    "moe_token_logprobs_backward", "moe_dropout", "moe_rms_norm", "moe_rms_norm_workspace_bytes",
    "moe_rms_norm_backward", "moe_grad_norm_workspace_bytes", "moe_grad_norm", "moe_adamw",
)


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_name(status)} ({status})")


class Shape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int),
                ("E", ctypes.c_int), ("k", ctypes.c_int), ("S", ctypes.c_int),
                ("dtype", ctypes.c_int)]

    @classmethod
    def of(cls, w: Workload) -> "Shape":
        return cls(w.N, w.H, w.I, w.E, w.k, w.S, DTYPES[w.dtype])


class Params(ctypes.Structure):
    _fields_ = [("ring_slots", ctypes.c_int), ("minibatch", ctypes.c_int),
                ("gather_ctas", ctypes.c_int), ("compute_ctas", ctypes.c_int),
                ("timeout_ns", ctypes.c_longlong), ("test_skip_ready", ctypes.c_int),
                ("reverse_ring", ctypes.c_int)]


class Saved(ctypes.Structure):
    """moe_saved_t: device pointers of the activations the backward reads."""
    _fields_ = [("idx", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("inv", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("sched", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("uv", ctypes.c_void_p)]

    @classmethod
    def of(cls, t: dict) -> "Saved":
        """From a dict of tensors with the field names as keys."""
        return cls(*(t[f].data_ptr() for f, _ in cls._fields_))


class AdamWTensor(ctypes.Structure):
    """moe_adamw_tensor_t: one tensor of an optimiser's list."""
    _fields_ = [("param", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("state_dtype", ctypes.c_int), ("weight_decay", ctypes.c_float)]


class AdamWParams(ctypes.Structure):
    """moe_adamw_t: the parameters of one step."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64), ("seed", ctypes.c_uint64),
                ("device_lr", ctypes.c_void_p), ("device_step", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p)]


def load_library(path: str = _LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libmoe.so not built at {path}; run token_dispatch_expert_top_gb300.build")
    return ctypes.CDLL(path)


_lib = load_library()
_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_f32, _f64, _u64 = ctypes.c_float, ctypes.c_double, ctypes.c_uint64
_shp, _prm, _svd = ctypes.POINTER(Shape), ctypes.POINTER(Params), ctypes.POINTER(Saved)
_lst, _adw = ctypes.POINTER(AdamWTensor), ctypes.POINTER(AdamWParams)
_SIGS = {
    "moe_workspace_bytes": (_sz, [_shp, _prm]),
    "moe_workspace_init": (_i, [_vp, _sz, _vp]),
    "moe_last_device_status": (_i, [_vp, _vp]),
    "moe_status_string": (ctypes.c_char_p, [_i]),
    "moe_quantize_mxfp8": (_i, [_vp, _i, _i64, _i64, _vp, _vp, _vp]),
    "moe_quantize_nvfp4": (_i, [_vp, _i, _i64, _i64, _vp, _vp, _vp, _vp]),
    "moe_macro_workspace_bytes": (_sz, [_shp, _prm, _i]),
    "moe_forward_macrobatched": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _shp, _prm, _i, _vp, _vp, _sz, _vp]),
    "moe_route_topk": (_i, [_vp, _vp, _vp, _shp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_layout": (_i, [_vp, _shp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_dispatch_pull": (_i, [_vp, _vp, _shp, _vp, _vp, _i, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "moe_expert_ffn": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _shp, _vp, _vp, _sz, _vp]),
    "moe_combine": (_i, [_vp, _vp, _vp, _shp, _vp, _vp, _sz, _vp]),
    "moe_forward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _shp, _prm, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_forward_fused": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _shp, _prm, _vp, _vp, _vp, _vp,
                               _sz, _vp]),
    "moe_min_minibatch": (_i, [_i, _i, _i, _i, _i]),
    "moe_layout_noalloc": (_i, [_vp, _shp, _vp, _vp, _vp, _vp, _vp]),
    "moe_pack_expert_weights": (_i, [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_backward_workspace_bytes": (_sz, [_shp]),
    "moe_pack_expert_weights_dgrad": (_i, [_shp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_expert_ffn_train": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _shp, _vp, _vp, _vp, _sz, _vp]),
    "moe_forward_train": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _shp, _prm, _vp, _svd, _vp, _sz,
                               _vp]),
    "moe_reverse_combine": (_i, [_vp, _vp, _vp, _vp, _shp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                 _vp]),
    "moe_expert_ffn_dgrad": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _shp, _vp, _vp, _vp, _vp,
                                  _vp, _sz, _vp]),
    "moe_reverse_dispatch": (_i, [_vp, _vp, _vp, _vp, _vp, _shp, _vp, _vp, _sz, _vp]),
    "moe_router_wgrad": (_i, [_vp, _vp, _vp, _vp, _shp, _vp, _vp, _vp, _sz, _vp]),
    "moe_backward": (_i, [_vp, _vp, _vp, _svd, _vp, _vp, _vp, _vp, _shp, _prm, _vp, _vp, _vp, _vp,
                          _vp, _vp, _sz, _vp]),
    "moe_expert_wgrad": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _shp, _vp, _vp, _vp, _sz, _vp]),
    "moe_embedding": (_i, [_vp, _i, _i64, _vp, _i, _i64, _i64, _i64, _f32, _vp, _i, _i64, _vp, _sz, _vp]),
    "moe_embedding_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "moe_embedding_backward": (_i, [_vp, _i, _i64, _i64, _i64, _vp, _i, _i64, _f32, _vp, _i, _i64, _i, _vp, _sz,
                                    _vp]),
    "moe_token_logprobs": (_i, [_vp, _i, _i64, _i64, _i64, _f32, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp, _sz,
                                _vp]),
    "moe_token_logprobs_backward": (_i, [_vp, _i, _i64, _i64, _i64, _f32, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i64,
                                         _vp, _sz, _vp]),
    "moe_dropout": (_i, [_vp, _i, _i64, _i64, _i64, _vp, _i64, _f64, _u64, _u64, _vp, _i64, _vp]),
    "moe_rms_norm": (_i, [_vp, _i, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i, _f32, _vp, _i, _i64, _vp, _vp,
                          _vp, _vp]),
    "moe_rms_norm_workspace_bytes": (_sz, [_i64, _i64]),
    "moe_rms_norm_backward": (_i, [_vp, _i, _i64, _i64, _i64, _vp, _i, _i64, _vp, _i, _vp, _vp, _i64, _vp, _i64, _vp,
                                   _i, _vp, _sz, _vp]),
    "moe_grad_norm_workspace_bytes": (_sz, []),
    "moe_grad_norm": (_i, [_lst, _i, _f32, _vp, _vp, _vp, _sz, _vp]),
    "moe_adamw": (_i, [_lst, _i, _adw, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def lib() -> ctypes.CDLL:
    return _lib


def status_name(code: int) -> str:
    return _lib.moe_status_string(code).decode()


def _p(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without building a torch.cuda.Stream around it (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(fn: str, rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(fn, rc)


# ------------------------------------------------------------------ entry points
def moe_workspace_bytes(shape: Shape, params: Params | None = None) -> int:
    return _lib.moe_workspace_bytes(ctypes.byref(shape), ctypes.byref(params) if params else None)


def moe_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check("moe_workspace_init", _lib.moe_workspace_init(_p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_last_device_status(ws: torch.Tensor, stream=None) -> int:
    return _lib.moe_last_device_status(_p(ws), _stream(stream))


def moe_status_string(code: int) -> str:
    return status_name(code)


def moe_quantize_mxfp8(inp: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    dt = MOE_BF16 if inp.dtype == torch.bfloat16 else MOE_F32
    K = inp.shape[-1]
    rows = inp.numel() // K
    _check("moe_quantize_mxfp8", _lib.moe_quantize_mxfp8(_p(inp), dt, rows, K, _p(codes), _p(scales),
                                                         _stream(stream)))


def moe_quantize_nvfp4(inp: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                       tensor_scale: torch.Tensor, stream=None) -> None:
    dt = MOE_BF16 if inp.dtype == torch.bfloat16 else MOE_F32
    K = inp.shape[-1]
    rows = inp.numel() // K
    _check("moe_quantize_nvfp4", _lib.moe_quantize_nvfp4(_p(inp), dt, rows, K, _p(codes), _p(scales),
                                                         _p(tensor_scale), _stream(stream)))


def moe_pack_expert_weights(shape: Shape, w_gate_up, w_gu_scales, w_down, w_d_scales,
                            packed_gate_up, packed_gu_scales, packed_down, packed_d_scales,
                            stream=None) -> None:
    _check("moe_pack_expert_weights", _lib.moe_pack_expert_weights(
        ctypes.byref(shape), _p(w_gate_up), _p(w_gu_scales), _p(w_down), _p(w_d_scales),
        _p(packed_gate_up), _p(packed_gu_scales), _p(packed_down), _p(packed_d_scales),
        _stream(stream)))


def _wsz(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def moe_route_topk(x, w_router, bias, shape: Shape, idx, gate, logits_out=None, xq_codes=None,
                   xq_scales=None, ws=None, stream=None) -> None:
    _check("moe_route_topk", _lib.moe_route_topk(
        _p(x), _p(w_router), _p(bias), ctypes.byref(shape), _p(idx), _p(gate), _p(logits_out),
        _p(xq_codes), _p(xq_scales), _p(ws), _wsz(ws), _stream(stream)))


def moe_layout(idx, shape: Shape, counts, offsets, sched, inv, ws, stream=None) -> None:
    _check("moe_layout", _lib.moe_layout(_p(idx), ctypes.byref(shape), _p(counts), _p(offsets),
                                         _p(sched), _p(inv), _p(ws), _wsz(ws), _stream(stream)))


def moe_dispatch_pull(shard_rows, shard_scales, shape: Shape, sched, inv, slot_begin: int,
                      slot_count: int, ring, ring_scales, ring_slots: int, ws, stream=None) -> None:
    """shard_rows / shard_scales: int64 device tensors holding S device pointers;
    inv: the [N][k] inverse map (visit slots token by token) or None (slot order)."""
    _check("moe_dispatch_pull", _lib.moe_dispatch_pull(
        _p(shard_rows), _p(shard_scales), ctypes.byref(shape), _p(sched), _p(inv), slot_begin,
        slot_count, _p(ring), _p(ring_scales), ring_slots, _p(ws), _wsz(ws), _stream(stream)))


def moe_expert_ffn(a, a_scales, offsets, w_gate_up, w_gu_scales, w_down, w_d_scales, shape: Shape,
                   y, ws, stream=None) -> None:
    _check("moe_expert_ffn", _lib.moe_expert_ffn(
        _p(a), _p(a_scales), _p(offsets), _p(w_gate_up), _p(w_gu_scales), _p(w_down),
        _p(w_d_scales), ctypes.byref(shape), _p(y), _p(ws), _wsz(ws), _stream(stream)))


def moe_combine(y, inv, gate, shape: Shape, out, ws, stream=None) -> None:
    _check("moe_combine", _lib.moe_combine(_p(y), _p(inv), _p(gate), ctypes.byref(shape), _p(out),
                                           _p(ws), _wsz(ws), _stream(stream)))


def moe_forward(x, w_router, bias, w_gate_up, w_gu_scales, w_down, w_d_scales, shape: Shape,
                params: Params | None, out, idx_out, gate_out, ws, stream=None) -> None:
    _check("moe_forward", _lib.moe_forward(
        _p(x), _p(w_router), _p(bias), _p(w_gate_up), _p(w_gu_scales), _p(w_down), _p(w_d_scales),
        ctypes.byref(shape), ctypes.byref(params) if params else None, _p(out), _p(idx_out),
        _p(gate_out), _p(ws), _wsz(ws), _stream(stream)))


def moe_macro_workspace_bytes(shape: Shape, params: Params | None, macrobatches: int) -> int:
    return _lib.moe_macro_workspace_bytes(ctypes.byref(shape), ctypes.byref(params) if params else None,
                                          macrobatches)


def moe_forward_macrobatched(x, w_router, bias, w_gate_up, w_gu_scales, w_down, w_d_scales, shape: Shape,
                             params: Params | None, macrobatches: int, out, ws, stream=None) -> None:
    _check("moe_forward_macrobatched", _lib.moe_forward_macrobatched(
        _p(x), _p(w_router), _p(bias), _p(w_gate_up), _p(w_gu_scales), _p(w_down), _p(w_d_scales),
        ctypes.byref(shape), ctypes.byref(params) if params else None, macrobatches, _p(out), _p(ws),
        _wsz(ws), _stream(stream)))


def moe_forward_fused(x, w_router, bias, w_gate_up, w_gu_scales, w_down, w_d_scales, shape: Shape,
                      params: Params | None, out, idx_out, gate_out, ws, stream=None) -> None:
    _check("moe_forward_fused", _lib.moe_forward_fused(
        _p(x), _p(w_router), _p(bias), _p(w_gate_up), _p(w_gu_scales), _p(w_down), _p(w_d_scales),
        ctypes.byref(shape), ctypes.byref(params) if params else None, _p(out), _p(idx_out),
        _p(gate_out), _p(ws), _wsz(ws), _stream(stream)))


def moe_min_minibatch(waves: int, compute_sms: int, tile_m: int, tile_n: int, I: int) -> int:
    return _lib.moe_min_minibatch(waves, compute_sms, tile_m, tile_n, I)


def moe_layout_noalloc(idx, shape: Shape, counts, offsets, sched, inv, stream=None) -> None:
    """moe_layout for callers that cannot allocate: no workspace argument; the
    library's fixed device scratch array is used instead (see include/moe.h)."""
    _check("moe_layout_noalloc", _lib.moe_layout_noalloc(
        _p(idx), ctypes.byref(shape), _p(counts), _p(offsets), _p(sched), _p(inv), _stream(stream)))


# ------------------------------------------------------------------ backward
def moe_backward_workspace_bytes(shape: Shape) -> int:
    return _lib.moe_backward_workspace_bytes(ctypes.byref(shape))


def moe_pack_expert_weights_dgrad(shape: Shape, w_gate_up, w_down, packed_gate_up_t,
                                  packed_gu_t_scales, packed_down_t, packed_d_t_scales,
                                  stream=None) -> None:
    _check("moe_pack_expert_weights_dgrad", _lib.moe_pack_expert_weights_dgrad(
        ctypes.byref(shape), _p(w_gate_up), _p(w_down), _p(packed_gate_up_t),
        _p(packed_gu_t_scales), _p(packed_down_t), _p(packed_d_t_scales), _stream(stream)))


def moe_expert_ffn_train(a, a_scales, offsets, w_gate_up, w_gu_scales, w_down, w_d_scales,
                         shape: Shape, y, uv, ws, stream=None) -> None:
    _check("moe_expert_ffn_train", _lib.moe_expert_ffn_train(
        _p(a), _p(a_scales), _p(offsets), _p(w_gate_up), _p(w_gu_scales), _p(w_down),
        _p(w_d_scales), ctypes.byref(shape), _p(y), _p(uv), _p(ws), _wsz(ws), _stream(stream)))


def moe_forward_train(x, w_router, bias, w_gate_up, w_gu_scales, w_down, w_d_scales,
                      shape: Shape, params: Params | None, out, saved: Saved, ws,
                      stream=None) -> None:
    _check("moe_forward_train", _lib.moe_forward_train(
        _p(x), _p(w_router), _p(bias), _p(w_gate_up), _p(w_gu_scales), _p(w_down), _p(w_d_scales),
        ctypes.byref(shape), ctypes.byref(params) if params else None, _p(out),
        ctypes.byref(saved), _p(ws), _wsz(ws), _stream(stream)))


def moe_reverse_combine(dout, y, inv, gate, shape: Shape, dy, dy_scales, dgate, dlogit,
                        slot_gate, slot_dlogit, ws, stream=None) -> None:
    _check("moe_reverse_combine", _lib.moe_reverse_combine(
        _p(dout), _p(y), _p(inv), _p(gate), ctypes.byref(shape), _p(dy), _p(dy_scales),
        _p(dgate), _p(dlogit), _p(slot_gate), _p(slot_dlogit), _p(ws), _wsz(ws), _stream(stream)))


def moe_expert_ffn_dgrad(dy, dy_scales, uv, offsets, wt_gate_up, wt_gu_scales, wt_down,
                         wt_d_scales, shape: Shape, duv, duv_codes, duv_scales, da, ws,
                         stream=None) -> None:
    _check("moe_expert_ffn_dgrad", _lib.moe_expert_ffn_dgrad(
        _p(dy), _p(dy_scales), _p(uv), _p(offsets), _p(wt_gate_up), _p(wt_gu_scales),
        _p(wt_down), _p(wt_d_scales), ctypes.byref(shape), _p(duv), _p(duv_codes),
        _p(duv_scales), _p(da), _p(ws), _wsz(ws), _stream(stream)))


def moe_reverse_dispatch(da, inv, idx, dlogit, w_router, shape: Shape, dx, ws, stream=None) -> None:
    _check("moe_reverse_dispatch", _lib.moe_reverse_dispatch(
        _p(da), _p(inv), _p(idx), _p(dlogit), _p(w_router), ctypes.byref(shape), _p(dx), _p(ws),
        _wsz(ws), _stream(stream)))


def moe_router_wgrad(x, sched, offsets, slot_dlogit, shape: Shape, dw_router, dbias, ws,
                     stream=None) -> None:
    _check("moe_router_wgrad", _lib.moe_router_wgrad(
        _p(x), _p(sched), _p(offsets), _p(slot_dlogit), ctypes.byref(shape), _p(dw_router),
        _p(dbias), _p(ws), _wsz(ws), _stream(stream)))


def moe_expert_wgrad(duv, x, dout, uv, sched, slot_gate, offsets, shape: Shape, dw_gate_up, dw_down,
                     ws, stream=None) -> None:
    _check("moe_expert_wgrad", _lib.moe_expert_wgrad(
        _p(duv), _p(x), _p(dout), _p(uv), _p(sched), _p(slot_gate), _p(offsets),
        ctypes.byref(shape), _p(dw_gate_up), _p(dw_down), _p(ws), _wsz(ws), _stream(stream)))


def moe_backward(dout, x, w_router, saved: Saved, wt_gate_up, wt_gu_scales, wt_down, wt_d_scales,
                 shape: Shape, params: Params | None, dx, dw_router, dbias, dw_gate_up, dw_down, ws,
                 stream=None) -> None:
    _check("moe_backward", _lib.moe_backward(
        _p(dout), _p(x), _p(w_router), ctypes.byref(saved), _p(wt_gate_up), _p(wt_gu_scales),
        _p(wt_down), _p(wt_d_scales), ctypes.byref(shape), ctypes.byref(params) if params else None,
        _p(dx), _p(dw_router), _p(dbias), _p(dw_gate_up), _p(dw_down), _p(ws), _wsz(ws),
        _stream(stream)))


# ------------------------------------------------------------------ operators around the layer
_FLOAT_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def _rows(fn: str, name: str, t: torch.Tensor) -> tuple[int, int, int, int, int]:
    """(pointer, moe dtype, rows, columns, row stride in elements) of a matrix whose rows
    are contiguous; leading dimensions that lie row after row count as rows."""
    dt = _FLOAT_DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{fn}: {name} is {t.dtype}; float32 or bfloat16 is wanted")
    if not t.is_cuda:
        raise ValueError(f"{fn}: {name} is not on a CUDA device")
    shape = t.shape
    if len(shape) != 2:
        if not shape:
            raise ValueError(f"{fn}: {name} has no columns")
        t = t.view(-1, shape[-1])
        shape = t.shape
    rows, cols = shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{fn}: the rows of {name} are not contiguous")
    return t.data_ptr(), dt, rows, cols, ld if rows > 1 else max(ld, cols)


def _ids(fn: str, name: str, t: torch.Tensor, n: int) -> tuple[int, int]:
    """(pointer, bytes per id) of n contiguous token ids."""
    size = _ID_BYTES.get(t.dtype)
    if size is None:
        raise TypeError(f"{fn}: {name} is {t.dtype}; int32 or int64 is wanted")
    _vector(fn, name, t, t.dtype, n)
    return t.data_ptr(), size


def _vector(fn: str, name: str, t: torch.Tensor, dtype: torch.dtype, n: int) -> None:
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{fn}: {name} has to be {n} contiguous elements of {dtype} on a CUDA device")


def moe_embedding(ids, table, out, scale: float = 1.0, ws=None, stream=None) -> None:
    """out[n] = scale * table[ids[n]]; out: [..., H], one row per id."""
    fn = "moe_embedding"
    tp, td, V, H, tl = _rows(fn, "table", table)
    op, od, N, oh, ol = _rows(fn, "out", out)
    if oh != H:
        raise ValueError(f"{fn}: out has {oh} columns, table {H}")
    ip, isz = _ids(fn, "ids", ids, N)
    _check(fn, _lib.moe_embedding(ip, isz, N, tp, td, V, H, tl, scale, op, od, ol, _p(ws), _wsz(ws),
                                  _stream(stream)))


def moe_embedding_workspace_bytes(N: int, V: int, H: int) -> int:
    return _lib.moe_embedding_workspace_bytes(N, V, H)


def moe_embedding_backward(ids, dout, dtable, scale: float = 1.0, accumulate: bool = False, ws=None,
                           stream=None) -> None:
    """dtable[v] (+)= scale * sum of dout's rows whose id is v."""
    fn = "moe_embedding_backward"
    gp, gd, N, gh, gl = _rows(fn, "dout", dout)
    tp, td, V, H, tl = _rows(fn, "dtable", dtable)
    if gh != H:
        raise ValueError(f"{fn}: dout has {gh} columns, dtable {H}")
    ip, isz = _ids(fn, "ids", ids, N)
    _check(fn, _lib.moe_embedding_backward(ip, isz, N, V, H, gp, gd, gl, scale, tp, td, tl, accumulate, _p(ws),
                                           _wsz(ws), _stream(stream)))


def moe_token_logprobs(logits, targets=None, logp=None, entropy=None, stats=None, top_idx=None, top_logp=None,
                       scale: float = 1.0, ws=None, stream=None) -> None:
    """Log probability of each row's target, entropy, the gradient's statistics and the
    top list, each into the tensor given for it (None: not computed)."""
    fn = "moe_token_logprobs"
    lp, dt, T, V, ld = _rows(fn, "logits", logits)
    tp, isz = (None, 4) if targets is None else _ids(fn, "targets", targets, T)
    n_top = 0
    if top_idx is not None and top_logp is not None:
        n_top = top_idx.shape[-1]
        _vector(fn, "top_idx", top_idx, torch.int32, T * n_top)
        _vector(fn, "top_logp", top_logp, torch.float32, T * n_top)
    elif top_idx is not None or top_logp is not None:
        raise ValueError(f"{fn}: top_idx and top_logp are given together")
    for name, t, n in (("logp", logp, T), ("entropy", entropy, T), ("stats", stats, 2 * T)):
        if t is not None:
            _vector(fn, name, t, torch.float32, n)
    _check(fn, _lib.moe_token_logprobs(lp, dt, T, V, ld, scale, tp, isz, _p(logp), _p(entropy), _p(stats), n_top,
                                       _p(top_idx) if n_top else None, _p(top_logp) if n_top else None, _p(ws),
                                       _wsz(ws), _stream(stream)))


def moe_token_logprobs_backward(logits, targets, stats, entropy, g_logp, g_entropy, dlogits, scale: float = 1.0,
                                ws=None, stream=None) -> None:
    """dlogits of moe_token_logprobs; dlogits may be logits itself."""
    fn = "moe_token_logprobs_backward"
    lp, dt, T, V, ld = _rows(fn, "logits", logits)
    dp, dd, dT, dV, dl = _rows(fn, "dlogits", dlogits)
    if (dd, dT, dV) != (dt, T, V):
        raise ValueError(f"{fn}: dlogits has to have logits' type and shape")
    tp, isz = (None, 4) if targets is None else _ids(fn, "targets", targets, T)
    for name, t, n in (("stats", stats, 2 * T), ("entropy", entropy, T), ("g_logp", g_logp, T),
                       ("g_entropy", g_entropy, T)):
        if t is not None:
            _vector(fn, name, t, torch.float32, n)
    _check(fn, _lib.moe_token_logprobs_backward(lp, dt, T, V, ld, scale, tp, isz, _p(stats), _p(entropy), _p(g_logp),
                                                _p(g_entropy), dp, dl, _p(ws), _wsz(ws), _stream(stream)))


def moe_dropout(x, out, p: float, seed: int, offset: int = 0, residual=None, stream=None) -> None:
    """out = residual + dropout(x); out may be x or residual."""
    fn = "moe_dropout"
    xp, dt, rows, cols, ld = _rows(fn, "x", x)
    op, od, orows, ocols, ol = _rows(fn, "out", out)
    rp, rl = None, 0
    if residual is not None:
        rp, rd, rrows, rcols, rl = _rows(fn, "residual", residual)
        if (rd, rrows, rcols) != (dt, rows, cols):
            raise ValueError(f"{fn}: residual has to have x's type and shape")
    if (od, orows, ocols) != (dt, rows, cols):
        raise ValueError(f"{fn}: out has to have x's type and shape")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError(f"{fn}: seed and offset are unsigned 64-bit numbers")
    _check(fn, _lib.moe_dropout(xp, dt, rows, cols, ld, rp, rl, p, seed, offset, op, ol, _stream(stream)))


# without the checks of torch.cuda.current_device, which a CUDA tensor has passed already
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_of(fn: str, name: str, t: torch.Tensor) -> int:
    """The device of a call's first tensor, which has to be the current one: the call goes to its stream."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{fn}: {name} is not on a CUDA device")
    if device != _current_device():
        raise ValueError(f"{fn}: {name} is on cuda:{device}, the current device is cuda:{_current_device()}")
    return device


def _stream_on(device: int, stream) -> int | None:
    return _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)


def _at(fn: str, name: str, t: torch.Tensor, dtype: torch.dtype, n: int, device: int) -> int:
    """The pointer of n contiguous elements of a type on that device."""
    if t.get_device() != device or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} has to be {n} contiguous elements of {dtype} on cuda:{device}")
    return t.data_ptr()


def _float_at(fn: str, name: str, t: torch.Tensor, n: int, device: int) -> tuple[int, int]:
    """(pointer, moe dtype) of n contiguous FP32 or BF16 elements on that device."""
    dt = _FLOAT_DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{fn}: {name} is {t.dtype}; float32 or bfloat16 is wanted")
    return _at(fn, name, t, t.dtype, n, device), dt


def _like(fn: str, name: str, t: torch.Tensor, other: str, want: tuple, device: int) -> tuple[int, int]:
    """(pointer, row stride) of a matrix of the type, rows and columns that `other` has, on its device."""
    p, dt, rows, cols, ld = _rows(fn, name, t)
    if (dt, rows, cols) != want:
        raise ValueError(f"{fn}: {name} has to have the type and shape of {other}")
    if t.get_device() != device:
        raise ValueError(f"{fn}: {name} is not on cuda:{device}")
    return p, ld


def moe_rms_norm(x, weight, out=None, eps: float = 1e-6, residual=None, sum=None, codes=None, scales=None, rstd=None,
                 stream=None) -> None:
    """out = s * weight / sqrt(mean(s^2) + eps) of each row, s = x or sum = x + residual; its MXFP8
    form into codes and scales, and the factor of each row into rstd, where they are given.  weight
    may be None, and out too if codes are given (they are then of x's type).  sum may be x or
    residual; without a residual out may be x."""
    fn = "moe_rms_norm"
    xp, dt, rows, cols, lx = _rows(fn, "x", x)
    device = _device_of(fn, "x", x)
    rp, rl, sp, sl, wp, wd = None, 0, None, 0, None, MOE_F32
    op, od, ol, cp, kp, tp = None, dt, 0, None, None, None
    if residual is not None and sum is not None:
        want = dt, rows, cols
        rp, rl = _like(fn, "residual", residual, "x", want, device)
        sp, sl = _like(fn, "sum", sum, "x", want, device)
    elif residual is not None or sum is not None:
        raise ValueError(f"{fn}: residual and sum are given together")
    if weight is not None:
        wp, wd = _float_at(fn, "weight", weight, cols, device)
    if out is not None:
        op, od, orows, ocols, ol = _rows(fn, "out", out)
        if orows != rows or ocols != cols or out.get_device() != device:
            raise ValueError(f"{fn}: out has to have x's shape and device")
    if codes is not None and scales is not None:
        if cols % 32:
            raise ValueError(f"{fn}: MXFP8 rows are whole blocks of 32; x has {cols} columns")
        cp = _at(fn, "codes", codes, torch.uint8, rows * cols, device)
        kp = _at(fn, "scales", scales, torch.uint8, rows * (cols // 32), device)
    elif codes is not None or scales is not None:
        raise ValueError(f"{fn}: codes and scales are given together")
    if rstd is not None:
        tp = _at(fn, "rstd", rstd, torch.float32, rows, device)
    rc = _lib.moe_rms_norm(xp, dt, rows, cols, lx, rp, rl, sp, sl, wp, wd, eps, op, od, ol, cp, kp, tp,
                           _stream_on(device, stream))
    if rc:
        raise MoeError(fn, rc)


def moe_rms_norm_workspace_bytes(rows: int, cols: int) -> int:
    return _lib.moe_rms_norm_workspace_bytes(rows, cols)


def moe_rms_norm_backward(dout, s, weight, rstd, dx, dweight=None, dsum=None, accumulate: bool = False, ws=None,
                          stream=None) -> None:
    """dx (the gradient of x and of residual alike, with dsum added) and dweight of moe_rms_norm; s:
    its sum, or x without a residual.  dx may be dsum, s or dout."""
    fn = "moe_rms_norm_backward"
    gp, gd, rows, cols, gl = _rows(fn, "dout", dout)
    device = _device_of(fn, "dout", dout)
    sp, dt, srows, scols, sl = _rows(fn, "s", s)
    if srows != rows or scols != cols or s.get_device() != device:
        raise ValueError(f"{fn}: s has to have dout's shape and device")
    want = dt, rows, cols
    xp, xl = _like(fn, "dx", dx, "s", want, device)
    up, ul, wp, wd, dp = None, 0, None, MOE_F32, None
    if dsum is not None:
        up, ul = _like(fn, "dsum", dsum, "s", want, device)
    if weight is not None:
        wp, wd = _float_at(fn, "weight", weight, cols, device)
    tp = _at(fn, "rstd", rstd, torch.float32, rows, device)
    if dweight is not None:
        dp = _at(fn, "dweight", dweight, torch.float32, cols, device)
    if ws is not None and ws.get_device() != device:
        raise ValueError(f"{fn}: ws is not on cuda:{device}")
    rc = _lib.moe_rms_norm_backward(gp, gd, rows, cols, gl, sp, dt, sl, wp, wd, tp, up, ul, xp, xl, dp, accumulate,
                                    _p(ws), _wsz(ws), _stream_on(device, stream))
    if rc:
        raise MoeError(fn, rc)


def _first_overlap(written: list, grads: list) -> str | None:
    """The first gradient (begin, bytes) that lies in one of the written ranges (begin, end, name), which are in
    order and apart, and the range's name."""
    begins = [begin for begin, _, _ in written]
    for i, (begin, size) in enumerate(grads):
        k = bisect_left(begins, begin + size) - 1             # the last one that begins before its end
        if size and k >= 0 and written[k][1] > begin:
            return f"grads[{i}] and {written[k][2]}"
    return None


class AdamWTensors:
    """The list of tensors that moe_adamw steps and moe_grad_norm measures, checked once and kept
    by a program beside its tensors (it holds on to them).

    params, grads, m, v: lists of contiguous CUDA tensors of one device, of the same number of
    elements place by place; params and grads FP32 or BF16.  m and v are FP32, or uint8 with
    m_scales and v_scales (lists of uint8, one per 32 elements; None at the places of FP32 moments)
    for moments in MXFP8.  copies: BF16 tensors, or None, which get each new weight.  weight_decay:
    one number, or one per tensor.  All but the gradients are written, and must not overlap; nor may a
    gradient lie in memory that is written, for moe_adamw (gradients may overlap each other)."""

    def __init__(self, params, grads, m, v, copies=None, m_scales=None, v_scales=None, weight_decay=0.0):
        fn, k = "AdamWTensors", len(params)
        none = [None] * k
        wd = [weight_decay] * k if isinstance(weight_decay, (int, float)) else weight_decay
        lists = dict(params=params, grads=grads, m=m, v=v, copies=copies if copies is not None else none,
                     m_scales=m_scales if m_scales is not None else none,
                     v_scales=v_scales if v_scales is not None else none, weight_decay=wd)
        for name, x in lists.items():
            if len(x) != k:
                raise ValueError(f"{fn}: {name} has {len(x)} entries, params {k}")
        self._kept = [list(x) for name, x in lists.items() if name != "grads"]
        self._start([p.numel() for p in params])
        for i, (e, p, m, v, copy, ms, vs, wd) in enumerate(zip(self.entries, *self._kept)):
            n = e.n
            e.param, e.param_dtype = self._float(f"params[{i}]", p, n)
            if m.dtype == torch.uint8:
                if ms is None or vs is None:
                    raise ValueError(f"{fn}: 8-bit moments come with m_scales and v_scales")
                e.state_dtype, state = MOE_MXFP8, torch.uint8
                e.m_scales = self._vector(f"m_scales[{i}]", ms, torch.uint8, (n + 31) // 32)
                e.v_scales = self._vector(f"v_scales[{i}]", vs, torch.uint8, (n + 31) // 32)
            else:
                e.state_dtype, state = MOE_F32, torch.float32
            e.m, e.v = self._vector(f"m[{i}]", m, state, n), self._vector(f"v[{i}]", v, state, n)
            if copy is not None:
                e.copy = self._vector(f"copies[{i}]", copy, torch.bfloat16, n)
            e.weight_decay = wd
        self._written = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), f"{name}[{i}]")
                               for name, x in lists.items() if name not in ("grads", "weight_decay")
                               for i, t in enumerate(x) if t is not None and t.numel())
        for (_, end, one), (begin, _, two) in zip(self._written, self._written[1:]):
            if begin < end:
                raise ValueError(f"{fn}: {one} and {two} overlap; memory that a step writes must not be there twice")
        self.set_grads(grads)

    @classmethod
    def of_grads(cls, grads) -> "AdamWTensors":
        """A list of gradients alone, for moe_grad_norm."""
        self = cls.__new__(cls)
        self._written = []
        self._start([g.numel() for g in grads])
        self.set_grads(grads)
        return self

    def _start(self, sizes):
        self.count, self.device, self._sizes = len(sizes), None, sizes
        self.entries = (AdamWTensor * max(1, self.count))()
        for e, n in zip(self.entries, sizes):
            e.n = n

    def _vector(self, name, t, dtype, n) -> int:
        if self.device is None:
            self.device = t.get_device()
            if self.device < 0:
                raise ValueError(f"AdamWTensors: {name} is not on a CUDA device")
        return _at("AdamWTensors", name, t, dtype, n, self.device)

    def _float(self, name, t, n) -> tuple[int, int]:
        dt = _FLOAT_DTYPES.get(t.dtype)
        if dt is None:
            raise TypeError(f"AdamWTensors: {name} is {t.dtype}; float32 or bfloat16 is wanted")
        return self._vector(name, t, t.dtype, n), dt

    def set_grads(self, grads) -> None:
        """Other tensors for the gradients, of the same sizes."""
        if len(grads) != self.count:
            raise ValueError(f"AdamWTensors: grads has {len(grads)} entries, not {self.count}")
        found = [self._float(f"grads[{i}]", g, n) for i, (n, g) in enumerate(zip(self._sizes, grads))]
        for e, (pointer, dtype) in zip(self.entries, found):
            e.grad, e.grad_dtype = pointer, dtype
        self._grads = list(grads)
        self._clash = _first_overlap(self._written, [(pointer, 4 * n if dtype == MOE_F32 else 2 * n)
                                                      for (pointer, dtype), n in zip(found, self._sizes)])


def _list_device(fn: str, tensors: AdamWTensors) -> int:
    """The list's device, which has to be the current one."""
    here = _current_device()
    if tensors.device is not None and tensors.device != here:
        raise ValueError(f"{fn}: the list's tensors are on cuda:{tensors.device}, the current device is cuda:{here}")
    return here


def moe_grad_norm_workspace_bytes() -> int:
    return _lib.moe_grad_norm_workspace_bytes()


def moe_grad_norm(tensors: AdamWTensors, norm=None, factor=None, max_norm: float = float("inf"), ws=None,
                  stream=None) -> None:
    """The norm of all gradients of the list, and the factor that brings it to max_norm at most (NaN
    if it is not finite), into FP32 tensors of one element."""
    fn = "moe_grad_norm"
    device = _list_device(fn, tensors)
    norm_at = None if norm is None else _at(fn, "norm", norm, torch.float32, 1, device)
    factor_at = None if factor is None else _at(fn, "factor", factor, torch.float32, 1, device)
    if ws is not None and ws.get_device() != device:
        raise ValueError(f"{fn}: ws is not on cuda:{device}")
    rc = _lib.moe_grad_norm(tensors.entries, tensors.count, max_norm, norm_at, factor_at, _p(ws), _wsz(ws),
                            _stream_on(device, stream))
    if rc:
        raise MoeError(fn, rc)


def moe_adamw(tensors: AdamWTensors, lr, step, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
              grad_scale=None, seed: int = 0, stream=None) -> None:
    """One AdamW step over the list.  lr: a number, or an FP32 tensor of one element; step: its number
    from 1, or an int64 tensor (tensors are read when the step runs: for CUDA graphs).  grad_scale:
    FP32 tensor that multiplies the gradients; if it is not finite nothing changes."""
    fn = "moe_adamw"
    if not 0 <= seed < 1 << 64:
        raise ValueError(f"{fn}: seed is an unsigned 64-bit number")
    device = _list_device(fn, tensors)
    if tensors._clash:
        raise ValueError(f"{fn}: {tensors._clash} overlap; a step must not write over the gradients it reads")
    lr_at, step_at, scale_at = None, None, None
    if isinstance(lr, torch.Tensor):
        lr, lr_at = 0.0, _at(fn, "lr", lr, torch.float32, 1, device)
    if isinstance(step, torch.Tensor):
        step, step_at = 0, _at(fn, "step", step, torch.int64, 1, device)
    if grad_scale is not None:
        scale_at = _at(fn, "grad_scale", grad_scale, torch.float32, 1, device)
    p = AdamWParams(lr, beta1, beta2, eps, step, seed, lr_at, step_at, scale_at)
    rc = _lib.moe_adamw(tensors.entries, tensors.count, p, _stream_on(device, stream))
    if rc:
        raise MoeError(fn, rc)
