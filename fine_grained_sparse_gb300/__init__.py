"""Fine-grained MoE layer forward (Kimi-K2 / Kimi-K3 shapes) on GB300.

A thin ctypes binding over the C ABI declared in ``include/moe.h``: every
function here has the C name, marshals tensors to pointers and raises
``MoeError`` on a non-zero status.  All arithmetic runs in the library's
CUDA kernels; there is no other implementation behind these names, and
importing the package fails when the library has not been built
(``python fine_grained_sparse_gb300/build.py``, or ``__graft_entry__.build()``).

Tensors are torch tensors on the current CUDA device (PyTorch provides the
device memory and the stream); plain integers are accepted as raw pointers.
"""
from __future__ import annotations

import bisect
import ctypes
import os
from typing import Optional, Sequence

from .build import lib_path

__all__ = [
    "MoeError", "MoeConfig", "MOE_F32", "MOE_BF16", "MOE_STAGE_COUNT", "STATUS", "lib",
    "config", "moe_version", "moe_status_string", "moe_validate_config", "moe_workspace_size",
    "moe_get_device_status", "moe_router", "moe_router_from_logits", "moe_permute",
    "moe_grouped_swiglu", "moe_combine", "moe_linear", "moe_layer_forward",
    "moe_layer_forward_host", "moe_layer_forward_host_pipelined", "moe_layer_forward_host_flush",
    "moe_layer_forward_host_release", "moe_last_error_detail",
    "moe_pack_weights", "pack_layer_weights",
    "moe_router_noalloc", "moe_launch_count", "moe_dense_gates", "moe_update_bias",
    "moe_quantile_bias_update",
    "MOE_WEIGHTS_NATURAL", "MOE_WEIGHTS_PACKED", "MOE_PACK_GATE_UP", "MOE_PACK_PLAIN",
    "MOE_WEIGHTS_PACKED_FP8", "moe_packed_fp8_bytes", "moe_pack_weights_fp8",
    "pack_layer_weights_fp8", "moe_selftest_bounded_wait", "MOE_ROUTER_WEIGHT_F32",
    "MOE_ROUTER_WEIGHT_SPLIT", "moe_router_weight_split_bytes", "moe_split_router_weight",
    "split_router_weight",
    "MOE_WEIGHTS_PACKED_INT4_G32", "MOE_WEIGHTS_PACKED_INT4_G128", "moe_packed_int4_bytes",
    "moe_pack_weights_int4", "pack_int4", "moe_grouped_swiglu_fp8_rows", "moe_linear_int4",
    "moe_add_rmsnorm", "moe_status_word",
    "moe_gather", "moe_combine_backward", "moe_router_backward", "moe_add_layernorm",
    "MOE_NORM_RMS", "MOE_NORM_LAYER", "moe_norm_backward", "moe_norm_backward_workspace_size",
    "AdamwTensor", "AdamwTable", "adamw_table", "moe_adamw",
]

MOE_F32, MOE_BF16 = 0, 1
MOE_WEIGHTS_NATURAL, MOE_WEIGHTS_PACKED, MOE_WEIGHTS_PACKED_FP8 = 0, 1, 2
MOE_WEIGHTS_PACKED_INT4_G32, MOE_WEIGHTS_PACKED_INT4_G128 = 3, 4
MOE_PACK_GATE_UP, MOE_PACK_PLAIN = 0, 1
MOE_ROUTER_WEIGHT_F32, MOE_ROUTER_WEIGHT_SPLIT = 0, 1
MOE_NORM_RMS, MOE_NORM_LAYER = 0, 1
MOE_STAGE_COUNT = 5
STAGE_NAMES = ("router", "dispatch", "expert_gate_up", "expert_down", "combine")
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
          3: "MOE_ERR_ALIGNMENT", 4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_CUDA",
          6: "MOE_ERR_TIMEOUT", 7: "MOE_ERR_DEVICE_INDEX"}


class MoeError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        self.status = status
        super().__init__(f"{func}: {STATUS.get(status, status)} ({detail})")


class MoeConfig(ctypes.Structure):
    _fields_ = [
        ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("E_routed", ctypes.c_int32),
        ("E_shared", ctypes.c_int32), ("d_ff_shared", ctypes.c_int32), ("K", ctypes.c_int32),
        ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
        ("routed_scaling_factor", ctypes.c_float), ("norm_topk_prob", ctypes.c_int32),
        ("d_latent", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("weight_layout", ctypes.c_int32), ("router_weight", ctypes.c_int32),
    ]


class AdamwTensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
        ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
        ("exp_avg_scale", ctypes.c_void_p), ("exp_avg_sq_scale", ctypes.c_void_p),
        ("n", ctypes.c_int64), ("weight_decay", ctypes.c_double),
    ]


def _load():
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError(
            f"fine_grained_sparse_gb300: CUDA library {path} is missing; build it with "
            "`python fine_grained_sparse_gb300/build.py`")
    return ctypes.CDLL(path)


lib = _load()

_P, _I32, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_D, _U64 = ctypes.c_double, ctypes.c_uint64
_CFG = ctypes.POINTER(MoeConfig)
_SIGS = {
    "moe_version": ([], _I32),
    "moe_launch_count": ([], ctypes.c_uint64),
    "moe_status_string": ([_I32], ctypes.c_char_p),
    "moe_last_error_detail": ([], ctypes.c_char_p),
    "moe_validate_config": ([_CFG, _I64], _I32),
    "moe_workspace_size": ([_CFG, _I64], _SZ),
    "moe_get_device_status": ([_P, _P], _I32),
    "moe_status_word": ([ctypes.POINTER(_P)], _I32),
    "moe_router": ([_CFG, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "moe_router_from_logits": ([_CFG, _I64, _P, _P, _P, _P, _P], _I32),
    "moe_dense_gates": ([_CFG, _I64, _P, _P, _P, _P], _I32),
    "moe_update_bias": ([_CFG, _I64, _P, _F, _P, _P], _I32),
    "moe_quantile_bias_update": ([_CFG, _I64, _P, _F, _P, _P, _P], _I32),
    "moe_permute": ([_CFG, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "moe_grouped_swiglu": ([_CFG, _I64] + [_P] * 12 + [_SZ, _P], _I32),
    "moe_combine": ([_CFG, _I64, _P, _P, _P, _P, _P, _P], _I32),
    "moe_linear": ([_I64, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "moe_pack_weights": ([_I32, _I64, _I64, _I64, _P, _P, _P], _I32),
    "moe_packed_fp8_bytes": ([_I64, _I64, _I64], _I64),
    "moe_selftest_bounded_wait": ([_P, _P], _I32),
    "moe_pack_weights_fp8": ([_I32, _I64, _I64, _I64, _P, _P, _P, _P], _I32),
    "moe_packed_int4_bytes": ([_I64, _I64, _I64, _I32], _I64),
    "moe_pack_weights_int4": ([_I32, _I64, _I64, _I64, _I32, _P, _P, _P, _P], _I32),
    "moe_grouped_swiglu_fp8_rows": ([_CFG, _I64] + [_P] * 14 + [_SZ, _P], _I32),
    "moe_linear_int4": ([_I64, _I32, _I32, _I32] + [_P] * 6, _I32),
    "moe_add_rmsnorm": ([_I32, _I64, _I32, _P, _P, _P, _F] + [_P] * 5, _I32),
    "moe_gather": ([_CFG, _I64] + [_P] * 6, _I32),
    "moe_combine_backward": ([_CFG, _I64] + [_P] * 7, _I32),
    "moe_router_backward": ([_CFG, _I64] + [_P] * 5, _I32),
    "moe_add_layernorm": ([_I32, _I64, _I32, _P, _P, _P, _P, _F, _P, _P, _P], _I32),
    "moe_norm_backward_workspace_size": ([_I64, _I32], _SZ),
    "moe_norm_backward": ([_I32, _I32, _I64, _I32, _P, _P, _P, _F] + [_P] * 6 + [_SZ, _P], _I32),
    "moe_adamw": ([_I32, _P, _I32, _I32, _I32, _D, _D, _D, _D, _I64, _P, _U64, _P], _I32),
    "moe_router_noalloc": ([_CFG, _I64, _P, _P, _P, _P, _P, _P], _I32),
    "moe_router_weight_split_bytes": ([_CFG], _SZ),
    "moe_split_router_weight": ([_CFG, _P, _P, _P], _I32),
    "moe_layer_forward": ([_CFG, _I64] + [_P] * 14 + [_SZ, _P, _P], _I32),
    "moe_layer_forward_host": ([_CFG, _I64] + [_P] * 11 + [_SZ, _P], _I32),
    "moe_layer_forward_host_pipelined": ([_CFG, _I64] + [_P] * 11 + [_SZ, _P], _I32),
    "moe_layer_forward_host_flush": ([_P, _P], _I32),
    "moe_layer_forward_host_release": ([_P], _I32),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    try:
        return t.data_ptr()
    except AttributeError:
        if type(t) is not int:  # a raw pointer; ctypes takes strings, bytes and booleans too
            raise
        return t


_current_stream = None  # () -> the current stream's handle, made on first use


def _make_current_stream():
    """The handle of torch's current stream.  A call of a few microseconds
    notices the Stream object that the public accessor builds, so the raw
    accessor is taken where torch has it."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    torch.cuda.current_stream()  # the accessors need an initialised context
    return lambda: raw(device())


def _stream(stream) -> Optional[int]:
    if stream is None:
        global _current_stream
        if _current_stream is None:
            _current_stream = _make_current_stream()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, func: str):
    if status != 0:
        raise MoeError(status, func, lib.moe_last_error_detail().decode())


def config(shape=None, **kw) -> MoeConfig:
    """MoeConfig from a ``synth.LayerShape``-like object and/or keywords."""
    vals = dict(d_model=0, d_ff=0, E_routed=0, E_shared=0, d_ff_shared=0, K=1, n_group=1,
                topk_group=1, routed_scaling_factor=2.827, norm_topk_prob=1, d_latent=0,
                dtype=MOE_BF16, weight_layout=MOE_WEIGHTS_NATURAL,
                router_weight=MOE_ROUTER_WEIGHT_F32)
    if shape is not None:
        for k in vals:
            if hasattr(shape, k):
                vals[k] = getattr(shape, k)
        if hasattr(shape, "dtype") and isinstance(shape.dtype, str):
            vals["dtype"] = MOE_F32 if shape.dtype == "f32" else MOE_BF16
        if getattr(shape, "router_only", False):
            vals["d_ff"] = 0
        if getattr(shape, "weights", "bf16") == "fp8":
            vals["weight_layout"] = MOE_WEIGHTS_PACKED_FP8
    vals.update(kw)
    vals["norm_topk_prob"] = int(bool(vals["norm_topk_prob"]))
    return MoeConfig(**vals)


def moe_version() -> int:
    return lib.moe_version()


def moe_launch_count() -> int:
    """Kernels the library has enqueued in this process so far."""
    return int(lib.moe_launch_count())


def moe_status_string(status: int) -> str:
    return lib.moe_status_string(status).decode()


def moe_last_error_detail() -> str:
    return lib.moe_last_error_detail().decode()


def moe_validate_config(cfg: MoeConfig, T: int) -> int:
    return lib.moe_validate_config(ctypes.byref(cfg), T)


def moe_workspace_size(cfg: MoeConfig, T: int) -> int:
    return lib.moe_workspace_size(ctypes.byref(cfg), T)


def moe_get_device_status(workspace, stream=None) -> int:
    return lib.moe_get_device_status(_ptr(workspace), _stream(stream))


def moe_status_word() -> int:
    """The address, on the current device, of the status word of calls without
    a workspace (moe_linear_int4), for moe_get_device_status."""
    word = _P()
    _check(lib.moe_status_word(ctypes.byref(word)), "moe_status_word")
    return word.value


def moe_router(cfg, T, x, W_r, bias, topk_idx, topk_w, workspace=None, ws_bytes=0, stream=None):
    _check(lib.moe_router(ctypes.byref(cfg), T, _ptr(x), _ptr(W_r), _ptr(bias), _ptr(topk_idx),
                          _ptr(topk_w), _ptr(workspace), ws_bytes, _stream(stream)), "moe_router")


def moe_dense_gates(cfg, T, topk_idx, topk_w, G, stream=None):
    """G [T, E] fp32: the routing weights at their experts, 0 elsewhere."""
    _check(lib.moe_dense_gates(ctypes.byref(cfg), T, _ptr(topk_idx), _ptr(topk_w), _ptr(G),
                               _stream(stream)), "moe_dense_gates")


def moe_update_bias(cfg, T, counts, gamma, bias, stream=None):
    """bias [E] fp32 in place: += gamma * sign(T K / E - counts)."""
    _check(lib.moe_update_bias(ctypes.byref(cfg), T, _ptr(counts), float(gamma), _ptr(bias),
                               _stream(stream)), "moe_update_bias")


def moe_quantile_bias_update(cfg, T, logits, rate, theta, bias, stream=None):
    """Quantile Balancing: theta [E] out, bias [E] fp32 updated in place."""
    _check(lib.moe_quantile_bias_update(ctypes.byref(cfg), T, _ptr(logits), float(rate),
                                        _ptr(theta), _ptr(bias), _stream(stream)),
           "moe_quantile_bias_update")


def moe_router_noalloc(cfg, T, x, W_r, bias, topk_idx, topk_w, stream=None):
    """moe_router on the library's static device scratch (no workspace)."""
    _check(lib.moe_router_noalloc(ctypes.byref(cfg), T, _ptr(x), _ptr(W_r), _ptr(bias),
                                  _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_router_noalloc")


def moe_router_from_logits(cfg, T, logits, bias, topk_idx, topk_w, stream=None):
    _check(lib.moe_router_from_logits(ctypes.byref(cfg), T, _ptr(logits), _ptr(bias),
                                      _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_router_from_logits")


def moe_permute(cfg, T, topk_idx, counts, offsets, perm, inv, workspace, ws_bytes, stream=None):
    _check(lib.moe_permute(ctypes.byref(cfg), T, _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                           _ptr(perm), _ptr(inv), _ptr(workspace), ws_bytes, _stream(stream)),
           "moe_permute")


def moe_grouped_swiglu(cfg, T, x_e, offsets, perm, topk_w, W_gate_up, W_down, x_shared,
                       Ws_gate_up, Ws_down, Y, Y_shared, workspace, ws_bytes, stream=None):
    _check(lib.moe_grouped_swiglu(ctypes.byref(cfg), T, _ptr(x_e), _ptr(offsets), _ptr(perm),
                                  _ptr(topk_w), _ptr(W_gate_up), _ptr(W_down), _ptr(x_shared),
                                  _ptr(Ws_gate_up), _ptr(Ws_down), _ptr(Y), _ptr(Y_shared),
                                  _ptr(workspace), ws_bytes, _stream(stream)),
           "moe_grouped_swiglu")


def moe_combine(cfg, T, Y, inv, topk_w, Y_shared, y, stream=None):
    """y = sum_k w_k Y[inv] + sum_s Y_shared; topk_w None means weight 1 (the
    weights already in Y)."""
    _check(lib.moe_combine(ctypes.byref(cfg), T, _ptr(Y), _ptr(inv), _ptr(topk_w), _ptr(Y_shared),
                           _ptr(y), _stream(stream)), "moe_combine")


def moe_linear(T, in_features, out_features, x, W, add, y, workspace, ws_bytes, stream=None):
    _check(lib.moe_linear(T, in_features, out_features, _ptr(x), _ptr(W), _ptr(add), _ptr(y),
                          _ptr(workspace), ws_bytes, _stream(stream)), "moe_linear")


def moe_layer_forward(cfg, T, x, W_r, bias, W_gate_up, W_down, Ws_gate_up, Ws_down, W_lat_down,
                      W_lat_up, y, topk_idx_out=None, topk_w_out=None, counts_out=None,
                      workspace=None, ws_bytes=0, stage_events: Optional[Sequence] = None,
                      stream=None):
    ev_array = None
    if stage_events is not None:
        handles = []
        for e in stage_events:
            if e is None:  # this stage boundary is not recorded
                handles.append(None)
            elif hasattr(e, "cuda_event"):
                if not e.cuda_event:  # torch creates its events lazily, on first record
                    import torch
                    e.record(torch.cuda.current_stream() if stream is None else stream)
                handles.append(e.cuda_event)
            else:
                handles.append(int(e))
        if len(handles) != MOE_STAGE_COUNT + 1:
            raise ValueError("stage_events needs MOE_STAGE_COUNT + 1 events")
        ev_array = (ctypes.c_void_p * len(handles))(*handles)
    _check(lib.moe_layer_forward(ctypes.byref(cfg), T, _ptr(x), _ptr(W_r), _ptr(bias),
                                 _ptr(W_gate_up), _ptr(W_down), _ptr(Ws_gate_up), _ptr(Ws_down),
                                 _ptr(W_lat_down), _ptr(W_lat_up), _ptr(y), _ptr(topk_idx_out),
                                 _ptr(topk_w_out), _ptr(counts_out), _ptr(workspace), ws_bytes,
                                 ctypes.cast(ev_array, ctypes.c_void_p) if ev_array is not None else None,
                                 _stream(stream)), "moe_layer_forward")


def moe_layer_forward_host(cfg, T, x_host, W_r, bias, W_gate_up, W_down, Ws_gate_up, Ws_down,
                           W_lat_down, W_lat_up, y_host, workspace, ws_bytes, stream=None):
    _check(lib.moe_layer_forward_host(ctypes.byref(cfg), T, _ptr(x_host), _ptr(W_r), _ptr(bias),
                                      _ptr(W_gate_up), _ptr(W_down), _ptr(Ws_gate_up),
                                      _ptr(Ws_down), _ptr(W_lat_down), _ptr(W_lat_up),
                                      _ptr(y_host), _ptr(workspace), ws_bytes, _stream(stream)),
           "moe_layer_forward_host")


def moe_layer_forward_host_pipelined(cfg, T, x_host, W_r, bias, W_gate_up, W_down, Ws_gate_up,
                                     Ws_down, W_lat_down, W_lat_up, y_host, workspace, ws_bytes,
                                     stream=None):
    """moe_layer_forward_host whose y_host is valid once `stream` has passed
    the next such call on the workspace, or moe_layer_forward_host_flush."""
    _check(lib.moe_layer_forward_host_pipelined(
        ctypes.byref(cfg), T, _ptr(x_host), _ptr(W_r), _ptr(bias), _ptr(W_gate_up), _ptr(W_down),
        _ptr(Ws_gate_up), _ptr(Ws_down), _ptr(W_lat_down), _ptr(W_lat_up), _ptr(y_host),
        _ptr(workspace), ws_bytes, _stream(stream)), "moe_layer_forward_host_pipelined")


def moe_layer_forward_host_flush(workspace, stream=None):
    """Make `stream` wait for the latest pipelined call's copy of y."""
    _check(lib.moe_layer_forward_host_flush(_ptr(workspace), _stream(stream)),
           "moe_layer_forward_host_flush")


def moe_layer_forward_host_release(workspace):
    """Drop the library's per-workspace state of moe_layer_forward_host."""
    _check(lib.moe_layer_forward_host_release(_ptr(workspace)), "moe_layer_forward_host_release")


def moe_pack_weights(kind, groups, rows, cols, src, dst, stream=None):
    _check(lib.moe_pack_weights(kind, groups, rows, cols, _ptr(src), _ptr(dst), _stream(stream)),
           "moe_pack_weights")


def moe_router_weight_split_bytes(cfg) -> int:
    return int(lib.moe_router_weight_split_bytes(ctypes.byref(cfg)))


def moe_split_router_weight(cfg, W_r, W_split, stream=None):
    _check(lib.moe_split_router_weight(ctypes.byref(cfg), _ptr(W_r), _ptr(W_split),
                                       _stream(stream)), "moe_split_router_weight")


def split_router_weight(cfg, W_r, stream=None):
    """The MOE_ROUTER_WEIGHT_SPLIT form of an fp32 router weight on W_r's
    device: a new bf16 [E, 3 d] tensor, for a config whose router_weight is
    MOE_ROUTER_WEIGHT_SPLIT (a one-time load step)."""
    import torch
    out = torch.empty((cfg.E_routed, 3 * cfg.d_model), dtype=torch.bfloat16, device=W_r.device)
    moe_split_router_weight(cfg, W_r, out, stream)
    return out


def moe_selftest_bounded_wait(workspace, stream=None):
    """Enqueue one bounded device wait that runs out (about 2 s); the
    workspace status word then reads MOE_ERR_TIMEOUT."""
    _check(lib.moe_selftest_bounded_wait(_ptr(workspace), _stream(stream)),
           "moe_selftest_bounded_wait")


def moe_packed_fp8_bytes(groups, rows, cols) -> int:
    return int(lib.moe_packed_fp8_bytes(groups, rows, cols))


def moe_pack_weights_fp8(kind, groups, rows, cols, codes, scales, dst, stream=None):
    _check(lib.moe_pack_weights_fp8(kind, groups, rows, cols, _ptr(codes), _ptr(scales), _ptr(dst),
                                    _stream(stream)), "moe_pack_weights_fp8")


def pack_layer_weights_fp8(weights: dict, stream=None) -> dict:
    """The weights of one layer for a config whose weight_layout is
    MOE_WEIGHTS_PACKED_FP8: the FP8 banks (keys ``<bank>_q`` with codes and
    ``<bank>_s`` with block scales, as produced by ``synth.generate`` for an
    FP8 shape) packed into one uint8 buffer each under ``<bank>``, and the
    bf16 latent projections packed as by ``pack_layer_weights``."""
    import torch
    out = {k: v for k, v in weights.items() if not (k.endswith("_q") or k.endswith("_s"))}
    kinds = {"W_gate_up": MOE_PACK_GATE_UP, "Ws_gate_up": MOE_PACK_GATE_UP,
             "W_down": MOE_PACK_PLAIN, "Ws_down": MOE_PACK_PLAIN}
    for key, kind in kinds.items():
        q, sc = weights.get(key + "_q"), weights.get(key + "_s")
        if q is None:
            continue
        G, R, C = q.shape
        dst = torch.empty(moe_packed_fp8_bytes(G, R, C), dtype=torch.uint8, device=q.device)
        moe_pack_weights_fp8(kind, G, R, C, q.contiguous(), sc.contiguous(), dst, stream)
        out[key] = dst
    lat = {k: weights[k] for k in ("W_lat_down", "W_lat_up") if weights.get(k) is not None}
    if lat:
        out.update(pack_layer_weights(lat, stream))
    return out


def pack_layer_weights(weights: dict, stream=None) -> dict:
    """Copies of the bf16 weight banks of one layer (keys as produced by
    ``synth.generate``: W_gate_up, W_down, Ws_gate_up, Ws_down, W_lat_down,
    W_lat_up) in MOE_WEIGHTS_PACKED order; other entries are passed through.
    Use with a config whose weight_layout is MOE_WEIGHTS_PACKED."""
    import torch
    out = dict(weights)
    kinds = {"W_gate_up": MOE_PACK_GATE_UP, "Ws_gate_up": MOE_PACK_GATE_UP,
             "W_down": MOE_PACK_PLAIN, "Ws_down": MOE_PACK_PLAIN,
             "W_lat_down": MOE_PACK_PLAIN, "W_lat_up": MOE_PACK_PLAIN}
    for key, kind in kinds.items():
        w = weights.get(key)
        if w is None:
            continue
        w3 = w if w.dim() == 3 else w.unsqueeze(0)
        dst = torch.empty_like(w3)
        moe_pack_weights(kind, w3.shape[0], w3.shape[1], w3.shape[2], w3, dst, stream)
        out[key] = dst if w.dim() == 3 else dst.squeeze(0)
    return out


def moe_packed_int4_bytes(groups, rows, cols, group_size) -> int:
    return int(lib.moe_packed_int4_bytes(groups, rows, cols, group_size))


def moe_pack_weights_int4(kind, groups, rows, cols, group_size, codes, scales, dst, stream=None):
    _check(lib.moe_pack_weights_int4(kind, groups, rows, cols, group_size, _ptr(codes),
                                     _ptr(scales), _ptr(dst), _stream(stream)),
           "moe_pack_weights_int4")


def pack_int4(kind, codes, scales, stream=None):
    """One 4-bit bank packed into a new uint8 buffer: codes [G, rows, cols / 2]
    uint8 (two a byte, the even column low) and scales [G, rows, cols /
    group_size] bf16, on one GPU, kind as in moe_pack_weights (a one-time load
    step).  Raises ValueError for tensors of other types or shapes, MoeError
    for sizes that moe_pack_weights_int4 rejects.  A given stream waits for the
    current one, whose memory the result is."""
    import torch
    if codes.dtype != torch.uint8 or scales.dtype != torch.bfloat16:
        raise ValueError(f"pack_int4: uint8 codes and bfloat16 scales, not {codes.dtype} and "
                         f"{scales.dtype}")
    if (codes.dim() != 3 or scales.dim() != 3 or codes.shape[:2] != scales.shape[:2]
            or scales.shape[2] < 1 or 2 * codes.shape[2] % scales.shape[2]):
        raise ValueError(f"pack_int4: codes [G, rows, cols / 2] and scales [G, rows, cols / "
                         f"group_size], not {list(codes.shape)} and {list(scales.shape)}")
    if not codes.is_cuda or codes.device != scales.device:
        raise ValueError(f"pack_int4: codes and scales on one GPU, not {codes.device} and "
                         f"{scales.device}")
    G, R, C = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    group = C // scales.shape[2]
    dst = torch.empty(max(moe_packed_int4_bytes(G, R, C, group), 0), dtype=torch.uint8,
                      device=codes.device)
    codes, scales = codes.contiguous(), scales.contiguous()
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            handle = _stream(stream)
            stream = (torch.cuda.ExternalStream(handle, device=codes.device) if handle
                      else torch.cuda.default_stream(codes.device))
        stream.wait_stream(torch.cuda.current_stream(codes.device))
        for t in (codes, scales, dst):  # not handed out again while the packing runs there
            t.record_stream(stream)
    moe_pack_weights_int4(kind, G, R, C, group, codes, scales, dst, stream)
    return dst


def moe_grouped_swiglu_fp8_rows(cfg, T, x_e, x_e_scale, offsets, perm, topk_w, W_gate_up, W_down,
                                x_shared, x_shared_scale, Ws_gate_up, Ws_down, Y, Y_shared,
                                workspace, ws_bytes, stream=None):
    """moe_grouped_swiglu on E4M3 rows with one fp32 scale per 128 columns (a
    4-bit weight layout)."""
    _check(lib.moe_grouped_swiglu_fp8_rows(
        ctypes.byref(cfg), T, _ptr(x_e), _ptr(x_e_scale), _ptr(offsets), _ptr(perm), _ptr(topk_w),
        _ptr(W_gate_up), _ptr(W_down), _ptr(x_shared), _ptr(x_shared_scale), _ptr(Ws_gate_up),
        _ptr(Ws_down), _ptr(Y), _ptr(Y_shared), _ptr(workspace), ws_bytes, _stream(stream)),
           "moe_grouped_swiglu_fp8_rows")


def moe_linear_int4(T, in_features, out_features, group_size, x, x_scale, W, add, y, stream=None):
    """y = x W^T (+ add) with a packed 4-bit W; x bf16, or E4M3 with x_scale."""
    _check(lib.moe_linear_int4(T, in_features, out_features, group_size, _ptr(x), _ptr(x_scale),
                               _ptr(W), _ptr(add), _ptr(y), _stream(stream)), "moe_linear_int4")


def moe_add_rmsnorm(dtype, T, d, x, residual, weight, eps, h, y, y_fp8=None, y_scale=None,
                    stream=None):
    """h = x + residual, y = weight * h / rms(h), in `dtype` and / or in E4M3
    with a scale per 128 columns."""
    _check(lib.moe_add_rmsnorm(dtype, T, d, _ptr(x), _ptr(residual), _ptr(weight), float(eps),
                               _ptr(h), _ptr(y), _ptr(y_fp8), _ptr(y_scale), _stream(stream)),
           "moe_add_rmsnorm")


def moe_gather(cfg, T, x, inv, topk_w, x_perm, w_perm=None, stream=None):
    """x_perm[inv] = x (and w_perm[inv] = topk_w): the rows in expert order."""
    _check(lib.moe_gather(ctypes.byref(cfg), T, _ptr(x), _ptr(inv), _ptr(topk_w), _ptr(x_perm),
                          _ptr(w_perm), _stream(stream)), "moe_gather")


def moe_combine_backward(cfg, T, dy, Y, inv, topk_w, dY, dtopk_w, stream=None):
    """dY[inv] = w dy and dtopk_w = <Y[inv], dy>: the gradient of moe_combine."""
    _check(lib.moe_combine_backward(ctypes.byref(cfg), T, _ptr(dy), _ptr(Y), _ptr(inv),
                                    _ptr(topk_w), _ptr(dY), _ptr(dtopk_w), _stream(stream)),
           "moe_combine_backward")


def moe_router_backward(cfg, T, logits, topk_idx, dtopk_w, dlogits, stream=None):
    """dlogits [T, E] of the gradient of the selected experts' weights."""
    _check(lib.moe_router_backward(ctypes.byref(cfg), T, _ptr(logits), _ptr(topk_idx),
                                   _ptr(dtopk_w), _ptr(dlogits), _stream(stream)),
           "moe_router_backward")


def moe_add_layernorm(dtype, T, d, x, residual, weight, bias, eps, h, y, stream=None):
    """h = x + residual, y = weight * (h - mean) / sqrt(var + eps) + bias."""
    _check(lib.moe_add_layernorm(dtype, T, d, _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias),
                                 float(eps), _ptr(h), _ptr(y), _stream(stream)),
           "moe_add_layernorm")


def moe_norm_backward_workspace_size(T, d) -> int:
    return int(lib.moe_norm_backward_workspace_size(T, d))


def moe_norm_backward(kind, dtype, T, d, x, residual, weight, eps, dy, dh, dx, dweight, dbias,
                      workspace=None, ws_bytes=0, stream=None):
    """The gradients of moe_add_rmsnorm (MOE_NORM_RMS) or moe_add_layernorm
    (MOE_NORM_LAYER): dx [T, d], dweight and dbias [d] fp32, each or None."""
    _check(lib.moe_norm_backward(kind, dtype, T, d, _ptr(x), _ptr(residual), _ptr(weight),
                                 float(eps), _ptr(dy), _ptr(dh), _ptr(dx), _ptr(dweight),
                                 _ptr(dbias), _ptr(workspace), ws_bytes, _stream(stream)),
           "moe_norm_backward")


class AdamwTable:
    """The tensors of moe_adamw, in the C layout; keeps them alive.  ``types``: the
    param_dtype, grad_dtype and state_bits that they are of, None without any.

    The table has the buffers' addresses: gradients must stay in theirs (backward
    into gradients that are there, ``zero_grad(set_to_none=False)``), or set_grads
    takes the new ones before the step."""

    def __init__(self, entries, tensors, types=(None, None, None), grads=(), written=()):
        self.entries, self.tensors, self.types = entries, tensors, types
        self.grads = list(grads)
        self._written = written  # (begin, end) of what the step writes, in order

    def __len__(self):
        return len(self.entries)

    def set_grads(self, grads) -> None:
        """``grads``, one for each of the table's tensors, in place of its gradients.
        Raises ValueError for what adamw_table refuses, or for another type; the
        table is then as it was.  Calls that were captured keep the old addresses."""
        grads = list(grads)
        if len(grads) != len(self.entries):
            raise ValueError(f"set_grads: {len(grads)} gradients of {len(self.entries)} tensors")
        device = self.tensors[0].device if self.tensors else None
        at = []
        for e, x in zip(self.entries, grads):
            if e.n == 0:
                at.append(None if x is None else x.data_ptr())
                continue
            if x is None or not x.is_cuda or not x.is_contiguous() or x.device != device:
                raise ValueError(f"set_grads: not a contiguous tensor on {device}")
            if x.numel() < e.n or _ADAMW_TYPES.get(str(x.dtype)) != self.types[1]:
                raise ValueError(f"set_grads: {x.numel()} elements of {x.dtype} for {e.n}")
            begin = x.data_ptr()
            i = bisect.bisect_left(self._written, (begin + e.n * x.element_size(),))
            if i and self._written[i - 1][1] > begin:
                raise ValueError("set_grads: a gradient overlaps a buffer that the step writes")
            at.append(begin)
        for e, a in zip(self.entries, at):
            e.grad = a
        self.grads = grads


_ADAMW_TYPES = {"torch.float32": MOE_F32, "torch.bfloat16": MOE_BF16}
_ADAMW_BITS = {"torch.float32": 32, "torch.uint8": 8, "torch.int8": 8, "torch.float8_e4m3fn": 8}


def adamw_table(tensors: Sequence[dict]) -> AdamwTable:
    """An AdamwTable of dicts with the fields of AdamwTensor: ``param``, ``grad``,
    ``exp_avg``, ``exp_avg_sq`` and, or None, ``master``, ``exp_avg_scale``,
    ``exp_avg_sq_scale`` (contiguous tensors on one GPU), ``n`` (param's size
    when missing) and ``weight_decay`` (0 when missing).  Params and gradients are
    float32 or bfloat16, the same for all, states float32 or codes (uint8, int8 or
    float8_e4m3fn), the same for all, the rest float32.  Raises ValueError for other types, for
    tensors that are not contiguous, on several devices, or smaller than n, and for
    a buffer that overlaps one that the step writes."""
    entries = (AdamwTensor * len(tensors))()
    device, keep, grads, ranges = None, [], [], []
    types = [None, None, None]
    for e, t in zip(entries, tensors):
        n = t.get("n")
        e.n = n = t["param"].numel() if n is None else int(n)
        e.weight_decay = float(t.get("weight_decay", 0.0))
        grads.append(t.get("grad"))
        for name in ("param", "grad", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                     "exp_avg_sq_scale"):
            x = t.get(name)
            if x is None:
                continue
            if not x.is_cuda or not x.is_contiguous():
                raise ValueError(f"adamw_table: {name} is not a contiguous tensor on a GPU")
            device = x.device if device is None else device
            need = -(-n // 128) if name.endswith("scale") else n
            if x.device != device or x.numel() < need:
                raise ValueError(f"adamw_table: {name} on {x.device} with {x.numel()} elements, "
                                 f"not on {device} with {need}")
            at = x.data_ptr()
            setattr(e, name, at)
            if name != "grad":
                keep.append(x)
            if n <= 0:
                continue
            dtype, slot = str(x.dtype), {"param": 0, "grad": 1, "exp_avg": 2, "exp_avg_sq": 2}.get(name)
            if slot is None:
                if dtype != "torch.float32":
                    raise ValueError(f"adamw_table: {name} is {dtype}, not torch.float32")
            else:
                kind = (_ADAMW_BITS if slot == 2 else _ADAMW_TYPES).get(dtype)
                if kind is None or types[slot] not in (None, kind):
                    raise ValueError(f"adamw_table: {name} of type {dtype}"
                                     + ("" if kind is None else " beside others"))
                types[slot] = kind
            ranges.append((at, at + need * x.element_size(), name))
    ranges.sort()
    written = read = 0  # the ends of what is written, and of all, up to here
    for at, end, name in ranges:
        if at < written or (at < read and name != "grad"):
            raise ValueError(f"adamw_table: {name} overlaps a buffer that is there already")
        read = max(read, end)
        if name != "grad":
            written = max(written, end)
    return AdamwTable(entries, keep, tuple(types), grads,
                      [(at, end) for at, end, name in ranges if name != "grad"])


def moe_adamw(table, param_dtype, grad_dtype, state_bits, lr, beta1, beta2, eps, step,
              grad_scale=None, seed=None, stream=None):
    """One AdamW step over the tensors of an AdamwTable.  Raises ValueError where
    their types are others than the call's.  ``seed``: of 8-bit states' random
    roundings, another in every step; the step's number when missing (the same bits in
    every step would hold a moment where it is)."""
    given = (param_dtype, grad_dtype, state_bits)
    if table.types != given and any(a not in (None, b) for a, b in zip(table.types, given)):
        raise ValueError(f"moe_adamw: types (param_dtype, grad_dtype, state_bits) {given} for a "
                         f"table of {table.types}")
    _check(lib.moe_adamw(len(table), ctypes.addressof(table.entries), param_dtype, grad_dtype,
                         state_bits, lr, beta1, beta2, eps, step, _ptr(grad_scale),
                         step if seed is None else seed, _stream(stream)), "moe_adamw")
