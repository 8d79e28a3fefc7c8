"""ctypes binding of libmoe_gb300.so: argument marshalling only.

Every function here allocates its outputs with torch on the inputs' device,
passes raw pointers, sizes and the current CUDA stream to the C entry point
of the same name, and raises MoEError on a non-OK status.  All arithmetic
runs in the library's CUDA kernels.  There is no fallback: if the library
is missing, importing this module fails.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_CUDA",
                4: "MOE_ERR_TIMEOUT", 5: "MOE_ERR_BAD_INDEX", 6: "MOE_ERR_WORKSPACE", 7: "MOE_ERR_NO_DEVICE"}


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {detail}")
        self.status = status


class ForwardLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("topk_idx", "topk_w", "counts", "offsets", "src_token", "dest_row", "row_w",
                 "x_perm", "h", "y", "total")]


class AdamWTensor(ctypes.Structure):
    """moe_adamw_tensor_t: one tensor of an optimizer list (device pointers)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64), ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32),
        ("state_bits", ctypes.c_int32), ("decay", ctypes.c_float)]


class AdamWHyper(ctypes.Structure):
    """moe_adamw_hyper_t: the coefficients of one step."""
    _fields_ = [(n, ctypes.c_float) for n in
                ("beta1", "one_minus_beta1", "beta2", "one_minus_beta2", "step_size", "decay", "inv_sqrt_bias", "eps")]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run sparse_expert_gb300/build.py (nvcc, sm_103a)")

lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_D = ctypes.c_double
_S = ctypes.c_int  # moe_status_t

SIGNATURES = {
    "moe_abi_version": (ctypes.c_int, []),
    "moe_status_string": (ctypes.c_char_p, [_S]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_route_topk": (_S, [_P, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "moe_route_topk_grouped": (_S, [_P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "moe_router_packed_bytes": (_SZ, [_I32, _I32]),
    "moe_pack_router_weights": (_S, [_P, _I32, _I32, _P, _P]),
    "moe_router_topk": (_S, [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _SZ, _P]),
    "moe_forward_routed": (_S, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "moe_dispatch_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "moe_dispatch_scan": (_S, [_P, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_dispatch_scan_noalloc": (_S, [_P, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P]),
    "moe_permute": (_S, [_P, _I64, _I32, _P, _I32, _P, _P]),
    "moe_packed_weight_bytes": (_SZ, [_I32, _I32, _I32]),
    "moe_pack_weights": (_S, [_P, _P, _P, _I32, _I32, _I32, _P, _P]),
    "moe_quantize_fp8_blockwise": (_S, [_P, _I64, _P, _P, _P]),
    "moe_dequantize_fp8_blockwise": (_S, [_P, _P, _I64, _P, _P]),
    "moe_fp8_packed_weight_bytes": (_SZ, [_I32, _I32, _I32]),
    "moe_pack_weights_fp8": (_S, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P]),
    "moe_forward_fp8": (_S, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "moe_forward_fp8_timed": (_S, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _SZ, _P, _P]),
    "moe_grouped_swiglu_workspace_bytes": (_SZ, []),
    "moe_grouped_swiglu": (_S, [_P, _P, _I64, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_combine": (_S, [_P, _P, _P, _I64, _I32, _I32, _P, _P]),
    "moe_combine_backward": (_S, [_P, _P, _P, _P, _I64, _I32, _I32, _P, _P, _P]),
    "moe_route_backward": (_S, [_P, _P, _P, _I64, _I32, _I32, _I32, _P, _P]),
    "moe_forward_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
    "moe_forward_layout": (_S, [_I64, _I32, _I32, _I32, _I32, ctypes.POINTER(ForwardLayout)]),
    "moe_forward": (_S, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "moe_forward_timed": (_S, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _SZ, _P, _P]),
    "moe_forward_gathered": (_S, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "moe_forward_gathered_timed": (_S, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _SZ, _P, _P]),
    "moe_forward_host": (_S, [_P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _SZ, _P]),
    "moe_read_device_status": (_S, [_P, _P, ctypes.POINTER(_I32)]),
    "moe_get_device_status": (_S, [_P, _P]),
    "moe_dispatch_noalloc_status": (_S, [_P, ctypes.POINTER(_I32)]),
    "moe_selftest_wait_timeout": (_S, [_P, _SZ, _I64, _P]),
    "moe_selftest_steal_wait": (_S, [_P, _I64, _P]),
    "moe_selftest_activation": (_S, [_P, _I64, _P, _P, _P]),
    "moe_set_tile_schedule": (_S, [_I32]),
    "moe_occupy_sms": (_S, [_I32, _I64, _P]),
    "moe_forward_host_stream": (_S, [_P, _P, _P, _I32, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _SZ,
                                     _P, _P, _P]),
    "moe_grouped_gate_up_save": (_S, [_P, _P, _I64, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "moe_grouped_swiglu_backward": (_S, [_P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                         _SZ, _P]),
    "moe_backward_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
    "moe_backward": (_S, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_backward_timed": (_S, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P,
                                _P]),
    "moe_layer_norm": (_S, [_P, _I64, _P, _I64, _P, _P, _I64, _I32, _I32, _I32, _F, _P, _P, _P, _P]),
    "moe_layer_norm_backward_workspace_bytes": (_SZ, [_I64, _I32]),
    "moe_layer_norm_backward": (_S, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _I32, _I32, _I32, _P, _P, _P, _P, _SZ,
                                     _P]),
    "moe_router_loss_workspace_bytes": (_SZ, []),
    "moe_router_loss": (_S, [_P, _P, _P, _I64, _I32, _F, _F, _P, _P, _P, _P, _SZ, _P]),
    "moe_adamw_hyper": (_S, [_D, _D, _D, _D, _D, _I64, _P]),
    "moe_adamw_step": (_S, [_P, _I32, _P, _P, _P, _P]),
    "moe_grad_norm_workspace_bytes": (_SZ, []),
    "moe_grad_norm": (_S, [_P, _I32, _F, _P, _P, _SZ, _P]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoEError(status, where, lib.moe_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _event_handles(events, stream):
    """cudaEvent_t handles of torch events (None: no event at that boundary)."""
    for ev in events:
        if ev is not None and ev.cuda_event == 0:
            ev.record(stream)  # materialise the handle
    return (ctypes.c_void_p * len(events))(*[0 if ev is None else ev.cuda_event for ev in events])


def _contig(t, dtype, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def abi_version() -> int:
    return lib.moe_abi_version()


# --------------------------------------------------------------- stage 1
def moe_route_topk(logits, k, renormalize=True, n_groups=1, stream=None):
    """topk_idx int32 [T,k], topk_w fp32 [T,k] of fp32 router logits [T,E];
    n_groups > 1 takes k/n_groups experts from each group of consecutive experts."""
    _contig(logits, torch.float32, "logits")
    T, E = logits.shape
    idx = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    if n_groups == 1:
        _check(lib.moe_route_topk(_ptr(logits), T, E, k, int(bool(renormalize)), _ptr(idx), _ptr(w),
                                  _stream(stream)), "moe_route_topk")
    else:
        _check(lib.moe_route_topk_grouped(_ptr(logits), T, E, k, n_groups, int(bool(renormalize)), _ptr(idx),
                                          _ptr(w), _stream(stream)), "moe_route_topk_grouped")
    return idx, w


def moe_pack_router_weights(w_router, stream=None):
    """Router weights [d, E] bf16 in the fused router's layout (uint8 buffer)."""
    _contig(w_router, torch.bfloat16, "w_router")
    d, E = w_router.shape
    packed = torch.empty(lib.moe_router_packed_bytes(d, E), dtype=torch.uint8, device=w_router.device)
    _check(lib.moe_pack_router_weights(_ptr(w_router), d, E, _ptr(packed), _stream(stream)), "moe_pack_router_weights")
    return packed


def moe_router_topk(x, router_packed, E, k, renormalize=True, stream=None):
    """Fused router: topk_idx [T,k], topk_w [T,k] of logits x @ w_router, never materialised."""
    _contig(x, torch.bfloat16, "x")
    T, d = x.shape
    idx = torch.empty(T, k, dtype=torch.int32, device=x.device)
    w = torch.empty(T, k, dtype=torch.float32, device=x.device)
    ws = torch.empty(256, dtype=torch.uint8, device=x.device)
    _check(lib.moe_router_topk(_ptr(x), _ptr(router_packed), T, d, E, k, int(bool(renormalize)), _ptr(idx), _ptr(w),
                               _ptr(ws), ws.numel(), _stream(stream)), "moe_router_topk")
    return idx, w


# ------------------------------------------------------------ stages 2-3
def moe_dispatch_workspace_bytes(T, E, k) -> int:
    return lib.moe_dispatch_workspace_bytes(T, E, k)


def moe_dispatch_scan(topk_idx, E, topk_w=None, row_w=True, workspace=None, stream=None):
    """counts [E], offsets [E+1], src_token [P], dest_row [P], row_w [P] (or None)."""
    _contig(topk_idx, torch.int32, "topk_idx")
    T, k = topk_idx.shape
    dev = topk_idx.device
    P = T * k
    if topk_w is not None:
        _contig(topk_w, torch.float32, "topk_w")
    need = lib.moe_dispatch_workspace_bytes(T, E, k)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    src = torch.empty(P, dtype=torch.int32, device=dev)
    dst = torch.empty(P, dtype=torch.int32, device=dev)
    rw = torch.empty(P, dtype=torch.float32, device=dev) if (row_w and topk_w is not None) else None
    _check(lib.moe_dispatch_scan(_ptr(topk_idx), _ptr(topk_w), T, E, k, _ptr(counts), _ptr(offsets), _ptr(src),
                                 _ptr(dst), _ptr(rw), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_dispatch_scan")
    return dict(counts=counts, offsets=offsets, src_token=src, dest_row=dst, row_w=rw, workspace=workspace)


def moe_dispatch_scan_noalloc(topk_idx, E, topk_w=None, row_w=True, stream=None):
    """moe_dispatch_scan without a workspace, for callers that cannot
    allocate device memory at call time (the library's fixed 4 MiB device
    scratch is used instead; overlapping calls race on it)."""
    _contig(topk_idx, torch.int32, "topk_idx")
    T, k = topk_idx.shape
    dev = topk_idx.device
    P = T * k
    if topk_w is not None:
        _contig(topk_w, torch.float32, "topk_w")
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    src = torch.empty(P, dtype=torch.int32, device=dev)
    dst = torch.empty(P, dtype=torch.int32, device=dev)
    rw = torch.empty(P, dtype=torch.float32, device=dev) if (row_w and topk_w is not None) else None
    _check(lib.moe_dispatch_scan_noalloc(_ptr(topk_idx), _ptr(topk_w), T, E, k, _ptr(counts), _ptr(offsets),
                                         _ptr(src), _ptr(dst), _ptr(rw), _stream(stream)),
           "moe_dispatch_scan_noalloc")
    return dict(counts=counts, offsets=offsets, src_token=src, dest_row=dst, row_w=rw)


# ---------------------------------------------------------- stage 4 / 5
def moe_permute(x, dest_row, k, stream=None):
    """x_perm [T*k, d] with x_perm[dest_row[t*k+j]] = x[t]."""
    _contig(x, torch.bfloat16, "x")
    _contig(dest_row, torch.int32, "dest_row")
    T, d = x.shape
    out = torch.empty(T * k, d, dtype=torch.bfloat16, device=x.device)
    _check(lib.moe_permute(_ptr(x), T, d, _ptr(dest_row), k, _ptr(out), _stream(stream)), "moe_permute")
    return out


def moe_packed_weight_bytes(E, d, f) -> int:
    return lib.moe_packed_weight_bytes(E, d, f)


def moe_pack_weights(w_gate, w_up, w_down, stream=None):
    """Packed expert weights (uint8 buffer) for moe_grouped_swiglu / moe_forward."""
    for t, n in ((w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        _contig(t, torch.bfloat16, n)
    E, d, f = w_gate.shape
    packed = torch.empty(lib.moe_packed_weight_bytes(E, d, f), dtype=torch.uint8, device=w_gate.device)
    _check(lib.moe_pack_weights(_ptr(w_gate), _ptr(w_up), _ptr(w_down), E, d, f, _ptr(packed), _stream(stream)),
           "moe_pack_weights")
    return packed


def moe_quantize_fp8_blockwise(w, stream=None):
    """(codes uint8 [n], scales fp32 [n/128]) of a bf16 tensor, blocks of 128 in memory order."""
    _contig(w, torch.bfloat16, "w")
    n = w.numel()
    codes = torch.empty(n, dtype=torch.uint8, device=w.device)
    scales = torch.empty(n // 128, dtype=torch.float32, device=w.device)
    _check(lib.moe_quantize_fp8_blockwise(_ptr(w), n, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_fp8_blockwise")
    return codes, scales


def moe_dequantize_fp8_blockwise(codes, scales, shape=None, stream=None):
    """bf16 weights (of ``shape``, flat by default) from codes and per-block scales."""
    _contig(codes, torch.uint8, "codes")
    _contig(scales, torch.float32, "scales")
    n = codes.numel()
    out = torch.empty(n, dtype=torch.bfloat16, device=codes.device)
    _check(lib.moe_dequantize_fp8_blockwise(_ptr(codes), _ptr(scales), n, _ptr(out), _stream(stream)),
           "moe_dequantize_fp8_blockwise")
    return out if shape is None else out.view(shape)


def moe_fp8_packed_weight_bytes(E, d, f) -> int:
    return lib.moe_fp8_packed_weight_bytes(E, d, f)


def moe_pack_weights_fp8(gate, up, down, E, d, f, stream=None):
    """FP8 weights (uint8 buffer) for moe_forward_fp8 from three (codes, scales)
    pairs as moe_quantize_fp8_blockwise returns them for w_gate, w_up [E,d,f]
    and w_down [E,f,d]."""
    for (c, sc), n in ((gate, "gate"), (up, "up"), (down, "down")):
        _contig(c, torch.uint8, n + " codes")
        _contig(sc, torch.float32, n + " scales")
    dev = gate[0].device
    packed = torch.empty(lib.moe_fp8_packed_weight_bytes(E, d, f), dtype=torch.uint8, device=dev)
    _check(lib.moe_pack_weights_fp8(_ptr(gate[0]), _ptr(gate[1]), _ptr(up[0]), _ptr(up[1]), _ptr(down[0]),
                                    _ptr(down[1]), E, d, f, _ptr(packed), _stream(stream)), "moe_pack_weights_fp8")
    return packed


def moe_forward_fp8(x, logits, packed_fp8, E, k, f, renormalize=True, workspace=None, out=None, topk_idx=None,
                    topk_w=None, stream=None):
    """moe_forward with FP8 weights packed by moe_pack_weights_fp8."""
    _contig(x, torch.bfloat16, "x")
    _contig(logits, torch.float32, "logits")
    T, d = x.shape
    dev = x.device
    if workspace is None:
        workspace = torch.empty(lib.moe_forward_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    _check(lib.moe_forward_fp8(_ptr(x), _ptr(logits), _ptr(packed_fp8), T, d, E, k, f, int(bool(renormalize)),
                               _ptr(out), _ptr(topk_idx), _ptr(topk_w), _ptr(workspace), workspace.numel(),
                               _stream(stream)),
           "moe_forward_fp8")
    return out


def moe_forward_fp8_timed(x, logits, packed_fp8, E, k, f, workspace, out, events, renormalize=True, stream=None):
    """moe_forward_fp8 recording events[0..6] at the stage boundaries."""
    T, d = x.shape
    s = stream if stream is not None else torch.cuda.current_stream()
    handles = _event_handles(events, s)
    _check(lib.moe_forward_fp8_timed(_ptr(x), _ptr(logits), _ptr(packed_fp8), T, d, E, k, f, int(bool(renormalize)),
                                     _ptr(out), _ptr(workspace), workspace.numel(), _stream(s), handles),
           "moe_forward_fp8_timed")
    return out


def moe_grouped_swiglu(x_perm, offsets, E, f, packed, row_scale=None, workspace=None, stream=None):
    """(h [P,f], y [P,d]) of the grouped SwiGLU expert MLP."""
    _contig(x_perm, torch.bfloat16, "x_perm")
    _contig(offsets, torch.int32, "offsets")
    P, d = x_perm.shape
    dev = x_perm.device
    if row_scale is not None:
        _contig(row_scale, torch.float32, "row_scale")
    if workspace is None:
        workspace = torch.empty(lib.moe_grouped_swiglu_workspace_bytes(), dtype=torch.uint8, device=dev)
    h = torch.empty(P, f, dtype=torch.bfloat16, device=dev)
    y = torch.empty(P, d, dtype=torch.bfloat16, device=dev)
    _check(lib.moe_grouped_swiglu(_ptr(x_perm), _ptr(offsets), P, E, d, f, _ptr(packed), _ptr(row_scale), _ptr(h),
                                  _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_grouped_swiglu")
    return h, y


def moe_grouped_gate_up_save(x_perm, offsets, E, f, packed, workspace=None, stream=None):
    """(h [P,f], gu [P,2f]): the gate/up GEMM keeping G and U, interleaved per gate/up tile."""
    _contig(x_perm, torch.bfloat16, "x_perm")
    _contig(offsets, torch.int32, "offsets")
    P, d = x_perm.shape
    dev = x_perm.device
    if workspace is None:
        workspace = torch.empty(lib.moe_grouped_swiglu_workspace_bytes(), dtype=torch.uint8, device=dev)
    h = torch.empty(P, f, dtype=torch.bfloat16, device=dev)
    gu = torch.empty(P, 2 * f, dtype=torch.bfloat16, device=dev)
    _check(lib.moe_grouped_gate_up_save(_ptr(x_perm), _ptr(offsets), P, E, d, f, _ptr(packed), _ptr(h), _ptr(gu),
                                        _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_grouped_gate_up_save")
    return h, gu


def gu_split(gu, f):
    """(G [P,f], U [P,f]) from the interleaved [P,2f] layout (a view reshuffle, for checks)."""
    h_t = 64
    t = gu.reshape(gu.shape[0], f // h_t, 2, h_t)
    return t[:, :, 0, :].reshape(gu.shape[0], f), t[:, :, 1, :].reshape(gu.shape[0], f)


def moe_grouped_swiglu_backward(x_perm, h, gu, dy, offsets, E, f, packed, workspace=None, stream=None):
    """dict(dgu, dx_perm, dw_gate, dw_up, dw_down) of the expert MLP backward."""
    for t, name in ((x_perm, "x_perm"), (h, "h"), (gu, "gu"), (dy, "dy")):
        _contig(t, torch.bfloat16, name)
    _contig(offsets, torch.int32, "offsets")
    P, d = x_perm.shape
    dev = x_perm.device
    if workspace is None:
        workspace = torch.empty(lib.moe_grouped_swiglu_workspace_bytes(), dtype=torch.uint8, device=dev)
    r = dict(dgu=torch.empty(P, 2 * f, dtype=torch.bfloat16, device=dev),
             dx_perm=torch.empty(P, d, dtype=torch.bfloat16, device=dev),
             dw_gate=torch.empty(E, d, f, dtype=torch.bfloat16, device=dev),
             dw_up=torch.empty(E, d, f, dtype=torch.bfloat16, device=dev),
             dw_down=torch.empty(E, f, d, dtype=torch.bfloat16, device=dev))
    _check(lib.moe_grouped_swiglu_backward(_ptr(x_perm), _ptr(h), _ptr(gu), _ptr(dy), _ptr(offsets), P, E, d, f,
                                           _ptr(packed), _ptr(r["dgu"]), _ptr(r["dx_perm"]), _ptr(r["dw_gate"]),
                                           _ptr(r["dw_up"]), _ptr(r["dw_down"]), _ptr(workspace), workspace.numel(),
                                           _stream(stream)),
           "moe_grouped_swiglu_backward")
    return r


def _backward_outputs(T, d, E, f, dev):
    return dict(dx=torch.empty(T, d, dtype=torch.bfloat16, device=dev),
                d_logits=torch.empty(T, E, dtype=torch.float32, device=dev),
                dw_gate=torch.empty(E, d, f, dtype=torch.bfloat16, device=dev),
                dw_up=torch.empty(E, d, f, dtype=torch.bfloat16, device=dev),
                dw_down=torch.empty(E, f, d, dtype=torch.bfloat16, device=dev))


def moe_backward(x, logits, packed, dout, E, k, f, renormalize=True, workspace=None, grads=None, stream=None):
    """dict(dx, d_logits, dw_gate, dw_up, dw_down): the layer backward (forward recomputed)."""
    _contig(x, torch.bfloat16, "x")
    _contig(logits, torch.float32, "logits")
    _contig(dout, torch.bfloat16, "dout")
    T, d = x.shape
    dev = x.device
    if workspace is None:
        workspace = torch.empty(lib.moe_backward_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device=dev)
    g = grads if grads is not None else _backward_outputs(T, d, E, f, dev)
    _check(lib.moe_backward(_ptr(x), _ptr(logits), _ptr(packed), _ptr(dout), T, d, E, k, f, int(bool(renormalize)),
                            _ptr(g["dx"]), _ptr(g["d_logits"]), _ptr(g["dw_gate"]), _ptr(g["dw_up"]),
                            _ptr(g["dw_down"]), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_backward")
    return g


BACKWARD_STAGES = ("recompute_route_index_permute", "recompute_gate_up", "output_grad_rows", "dgrad_down",
                   "dgrad_gate_up", "gate_grad_route_bwd", "wgrad_down", "wgrad_gate_up", "unpermute")


def moe_backward_timed(x, logits, packed, dout, E, k, f, workspace, grads, events, renormalize=True, stream=None):
    """moe_backward recording events[0..9] at the stage boundaries (BACKWARD_STAGES); a None entry records nothing."""
    T, d = x.shape
    s = stream if stream is not None else torch.cuda.current_stream()
    handles = _event_handles(events, s)
    g = grads
    _check(lib.moe_backward_timed(_ptr(x), _ptr(logits), _ptr(packed), _ptr(dout), T, d, E, k, f,
                                  int(bool(renormalize)), _ptr(g["dx"]), _ptr(g["d_logits"]), _ptr(g["dw_gate"]),
                                  _ptr(g["dw_up"]), _ptr(g["dw_down"]), _ptr(workspace), workspace.numel(), _stream(s),
                                  handles),
           "moe_backward_timed")
    return g


def moe_combine(y, dest_row, T, k, topk_w=None, stream=None):
    """out [T, d] = sum_j w[t,j] * y[dest_row[t*k+j]] (w = 1 when topk_w is None)."""
    _contig(y, torch.bfloat16, "y")
    _contig(dest_row, torch.int32, "dest_row")
    if topk_w is not None:
        _contig(topk_w, torch.float32, "topk_w")
    d = y.shape[1]
    out = torch.empty(T, d, dtype=torch.bfloat16, device=y.device)
    _check(lib.moe_combine(_ptr(y), _ptr(dest_row), _ptr(topk_w), T, k, d, _ptr(out), _stream(stream)),
           "moe_combine")
    return out


def moe_combine_backward(dout, mlp_out, dest_row, topk_w, stream=None):
    """(d_mlp_out [T*k, d] bf16, d_topk_w [T, k] fp32) of the output reduction."""
    _contig(dout, torch.bfloat16, "dout")
    _contig(mlp_out, torch.bfloat16, "mlp_out")
    _contig(dest_row, torch.int32, "dest_row")
    _contig(topk_w, torch.float32, "topk_w")
    T, d = dout.shape
    k = topk_w.shape[1]
    dy = torch.empty(T * k, d, dtype=torch.bfloat16, device=dout.device)
    dw = torch.empty(T, k, dtype=torch.float32, device=dout.device)
    _check(lib.moe_combine_backward(_ptr(dout), _ptr(mlp_out), _ptr(dest_row), _ptr(topk_w), T, k, d, _ptr(dy),
                                    _ptr(dw), _stream(stream)), "moe_combine_backward")
    return dy, dw


def moe_route_backward(logits, topk_idx, d_topk_w, renormalize=True, stream=None):
    """d_logits [T, E] fp32 from the gates' gradient (selection held fixed)."""
    _contig(logits, torch.float32, "logits")
    _contig(topk_idx, torch.int32, "topk_idx")
    _contig(d_topk_w, torch.float32, "d_topk_w")
    T, E = logits.shape
    k = topk_idx.shape[1]
    out = torch.empty(T, E, dtype=torch.float32, device=logits.device)
    _check(lib.moe_route_backward(_ptr(logits), _ptr(topk_idx), _ptr(d_topk_w), T, E, k, int(bool(renormalize)),
                                  _ptr(out), _stream(stream)), "moe_route_backward")
    return out


# ------------------------------------------------------------ the layer
def moe_forward_workspace_bytes(T, E, k, d, f) -> int:
    return lib.moe_forward_workspace_bytes(T, E, k, d, f)


def moe_backward_workspace_bytes(T, E, k, d, f) -> int:
    return lib.moe_backward_workspace_bytes(T, E, k, d, f)


def moe_forward_layout(T, E, k, d, f) -> ForwardLayout:
    lay = ForwardLayout()
    _check(lib.moe_forward_layout(T, E, k, d, f, ctypes.byref(lay)), "moe_forward_layout")
    return lay


def moe_forward(x, logits, packed, E, k, f, renormalize=True, workspace=None, out=None, topk_idx=None,
                topk_w=None, stream=None):
    """out [T, d] of the whole layer.  The workspace keeps every intermediate."""
    _contig(x, torch.bfloat16, "x")
    _contig(logits, torch.float32, "logits")
    T, d = x.shape
    dev = x.device
    if workspace is None:
        workspace = torch.empty(lib.moe_forward_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    _check(lib.moe_forward(_ptr(x), _ptr(logits), _ptr(packed), T, d, E, k, f, int(bool(renormalize)), _ptr(out),
                           _ptr(topk_idx), _ptr(topk_w), _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_forward")
    return out


FORWARD_STAGES = ("route", "index", "permute", "gate_up", "down", "combine")


def moe_forward_gathered(x, logits, packed, E, k, f, renormalize=True, workspace=None, out=None, topk_idx=None,
                         topk_w=None, stream=None):
    """moe_forward with the gate/up GEMM gathering its rows from x (no x_perm)."""
    _contig(x, torch.bfloat16, "x")
    _contig(logits, torch.float32, "logits")
    T, d = x.shape
    dev = x.device
    if workspace is None:
        workspace = torch.empty(lib.moe_forward_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    _check(lib.moe_forward_gathered(_ptr(x), _ptr(logits), _ptr(packed), T, d, E, k, f, int(bool(renormalize)),
                                    _ptr(out), _ptr(topk_idx), _ptr(topk_w), _ptr(workspace), workspace.numel(),
                                    _stream(stream)),
           "moe_forward_gathered")
    return out


def moe_forward_gathered_timed(x, logits, packed, E, k, f, workspace, out, events, renormalize=True, stream=None):
    """moe_forward_gathered recording events[0..6] at the stage boundaries."""
    T, d = x.shape
    s = stream if stream is not None else torch.cuda.current_stream()
    handles = _event_handles(events, s)
    _check(lib.moe_forward_gathered_timed(_ptr(x), _ptr(logits), _ptr(packed), T, d, E, k, f, int(bool(renormalize)),
                                          _ptr(out), _ptr(workspace), workspace.numel(), _stream(s), handles),
           "moe_forward_gathered_timed")
    return out


def moe_forward_routed(x, router_packed, packed, E, k, f, renormalize=True, workspace=None, out=None, stream=None):
    """out [T, d] of the whole layer from the tokens and the packed router weights."""
    _contig(x, torch.bfloat16, "x")
    T, d = x.shape
    dev = x.device
    if workspace is None:
        workspace = torch.empty(lib.moe_forward_workspace_bytes(T, E, k, d, f), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    _check(lib.moe_forward_routed(_ptr(x), _ptr(router_packed), _ptr(packed), T, d, E, k, f, int(bool(renormalize)),
                                  _ptr(out), None, None, _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_forward_routed")
    return out


def moe_forward_timed(x, logits, packed, E, k, f, workspace, out, events, renormalize=True, stream=None):
    """moe_forward that records events[0..6] (torch.cuda.Event, timing enabled)
    at the stage boundaries on the launching stream; a None entry records
    nothing at its boundary."""
    T, d = x.shape
    s = stream if stream is not None else torch.cuda.current_stream()
    handles = _event_handles(events, s)
    _check(lib.moe_forward_timed(_ptr(x), _ptr(logits), _ptr(packed), T, d, E, k, f, int(bool(renormalize)),
                                 _ptr(out), _ptr(workspace), workspace.numel(), _stream(s), handles),
           "moe_forward_timed")
    return out


def moe_forward_host(x_host, logits_host, out_host, x_dev, logits_dev, out_dev, packed, E, k, f, workspace,
                     renormalize=True, stream=None):
    """moe_forward from host tensors (pinned for full-speed copies); waits for the stream."""
    T, d = x_host.shape
    _check(lib.moe_forward_host(_ptr(x_host), _ptr(logits_host), _ptr(out_host), _ptr(x_dev), _ptr(logits_dev),
                                _ptr(out_dev), _ptr(packed), T, d, E, k, f, int(bool(renormalize)),
                                _ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_forward_host")
    return out_host


def moe_forward_host_stream(x_hosts, logits_hosts, out_hosts, x_dev, logits_dev, out_dev, packed, E, k, f,
                            workspace, renormalize=True, stream=None, copy_in=None, copy_out=None):
    """moe_forward over host batches with overlapped copies; *_dev are pairs of device slots."""
    n = len(x_hosts)
    T, d = x_hosts[0].shape
    stream = stream if stream is not None else torch.cuda.current_stream()
    copy_in = copy_in if copy_in is not None else torch.cuda.Stream()
    copy_out = copy_out if copy_out is not None else torch.cuda.Stream()

    def arr(ts):
        return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])
    _check(lib.moe_forward_host_stream(arr(x_hosts), arr(logits_hosts), arr(out_hosts), n, arr(x_dev),
                                       arr(logits_dev), arr(out_dev), _ptr(packed), T, d, E, k, f,
                                       int(bool(renormalize)), _ptr(workspace), workspace.numel(), _stream(stream),
                                       _stream(copy_in), _stream(copy_out)),
           "moe_forward_host_stream")
    return out_hosts


def moe_selftest_wait_timeout(workspace, limit_ns, stream=None):
    """Runs the bounded-wait check; read the status with moe_read_device_status."""
    _check(lib.moe_selftest_wait_timeout(_ptr(workspace), workspace.numel(), int(limit_ns), _stream(stream)),
           "moe_selftest_wait_timeout")


def moe_selftest_steal_wait(limit_ns, stream=None):
    """Outcomes [2, 128] of the block-wide wait: nothing comes, and it comes late."""
    out = torch.empty(2, 128, dtype=torch.int32, device="cuda")
    _check(lib.moe_selftest_steal_wait(_ptr(out), int(limit_ns), _stream(stream)), "moe_selftest_steal_wait")
    return out


def moe_selftest_activation(z, stream=None):
    """Silu(z) and sigmoid(z), fp32, computed by the device functions of the expert-GEMM epilogues."""
    z = _contig(z, torch.float32, "z")
    silu = torch.empty_like(z)
    sig = torch.empty_like(z)
    _check(lib.moe_selftest_activation(_ptr(z), z.numel(), _ptr(silu), _ptr(sig), _stream(stream)),
           "moe_selftest_activation")
    return silu, sig


TILE_SCHEDULE_DYNAMIC = 0
TILE_SCHEDULE_STATIC = 1


def moe_set_tile_schedule(mode):
    """The paired expert GEMMs' tile schedule for the rest of the process (measurement)."""
    _check(lib.moe_set_tile_schedule(int(mode)), "moe_set_tile_schedule")


def moe_occupy_sms(n_sms, duration_ns, stream=None):
    """A kernel holding n_sms SMs for duration_ns on `stream` (measurement)."""
    _check(lib.moe_occupy_sms(int(n_sms), int(duration_ns), _stream(stream)), "moe_occupy_sms")


def forward_intermediates(workspace, T, E, k, d, f):
    """Views of the intermediates that moe_forward leaves in its workspace."""
    lay = moe_forward_layout(T, E, k, d, f)
    P = T * k

    def view(off, n, dtype):
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return workspace[off:off + nbytes].view(dtype)
    return dict(
        counts=view(lay.counts, E, torch.int32),
        offsets=view(lay.offsets, E + 1, torch.int32),
        topk_idx=view(lay.topk_idx, P, torch.int32).view(T, k),
        topk_w=view(lay.topk_w, P, torch.float32).view(T, k),
        src_token=view(lay.src_token, P, torch.int32),
        dest_row=view(lay.dest_row, P, torch.int32),
        row_w=view(lay.row_w, P, torch.float32),
        x_perm=view(lay.x_perm, P * d, torch.bfloat16).view(P, d),
        h=view(lay.h, P * f, torch.bfloat16).view(P, f),
        y=view(lay.y, P * d, torch.bfloat16).view(P, d),
    )


def moe_read_device_status(workspace, stream=None) -> int:
    st = _I32(0)
    _check(lib.moe_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(st)), "moe_read_device_status")
    return st.value


def moe_get_device_status(workspace, stream=None) -> int:
    """The workspace's device status as the C call returns it (0 = MOE_OK,
    4 = MOE_ERR_TIMEOUT, 5 = MOE_ERR_BAD_INDEX); raises only when the read
    itself fails."""
    s = lib.moe_get_device_status(_ptr(workspace), _stream(stream))
    if s in (1, 3):  # MOE_ERR_INVALID_ARG, MOE_ERR_CUDA: the read failed
        _check(s, "moe_get_device_status")
    return s


def moe_dispatch_noalloc_status(stream=None) -> int:
    """Device status of the latest moe_dispatch_scan_noalloc on this device."""
    st = _I32(0)
    _check(lib.moe_dispatch_noalloc_status(_stream(stream), ctypes.byref(st)), "moe_dispatch_noalloc_status")
    return st.value


# ------------------------------------------- the training step around the layer
#
# These calls can be as short as their launch (a few microseconds), so their
# checks take the cheap accessors and look closer only where one fails.  With
# a stream argument everything runs under that stream, allocations included:
# memory taken from the current stream's pool could be handed out again there
# while the other stream's kernel still uses it.
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # moe_dtype_t
_raw_stream = torch._C._cuda_getCurrentRawStream  # cudaStream_t of the current stream of a device index
_current_device = torch._C._cuda_getDevice


def _elsewhere(t, name, index):
    """Raises for a tensor that is not on device `index`."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _here(index, name):
    """Raises unless device `index` is the one that the call launches on: the
    current device, or that of the call's stream."""
    if index != _current_device():
        raise ValueError(f"{name} must be on the current device (or the stream's), cuda:{_current_device()}, "
                         f"got cuda:{index}")


def _device_of(t, name):
    """Index of the device of a call's first operand, which the others share."""
    index = t.get_device()
    if index < 0:
        _elsewhere(t, name, index)
    _here(index, name)
    return index


def _workspace(t, index):
    """Bytes of a caller's workspace."""
    if t.get_device() != index:
        _elsewhere(t, "workspace", index)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.numel() * t.element_size()


def _rows(t, name, index, shape=None, dtype=None):
    """Checks a [T, d] tensor of rows (unit stride along d) and returns its row stride."""
    if t.get_device() != index:
        _elsewhere(t, name, index)
    if t.dtype is not dtype and (dtype is not None or t.dtype not in _DTYPES):
        raise TypeError(f"{name} must be {dtype or 'float32, bfloat16 or float16'}, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {'[T, d]' if shape is None else list(shape)}, got {list(t.shape)}")
    stride = t.stride()
    if stride[1] != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return stride[0]


def _norm_param(t, name, index, d, dtype):
    """Checks a weight or bias [d] and returns its moe_dtype_t."""
    wdt = t.dtype
    if wdt is not dtype and wdt is not torch.float32:
        raise TypeError(f"{name} must be float32 or {dtype}, got {wdt}")
    if t.shape != (d,):
        raise ValueError(f"{name} must be [{d}], got {list(t.shape)}")
    if t.get_device() != index:
        _elsewhere(t, name, index)
    if not t.is_contiguous():
        _contig(t, wdt, name)
    return _DTYPES[wdt]


def _out(t, index, shape, dtype, name):
    if t.get_device() != index:
        _elsewhere(t, name, index)
    if t.dtype is not dtype or not t.is_contiguous():
        _contig(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def moe_layer_norm(x, weight=None, bias=None, eps=1e-5, residual=None, out=None, stats=None, z=None, stream=None):
    """(y [T,d], stats [2,T]) of the rows of x [T,d] (any row stride), or
    (y, stats, z) with a residual: z = x + residual, y = layer norm of z.
    stats (mean, then reciprocal standard deviation) is what the backward reads."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_layer_norm(x, weight, bias, eps, residual, out, stats, z)
    index = _device_of(x, "x")
    x_stride = _rows(x, "x", index)
    shape, dt = x.shape, x.dtype
    T, d = shape
    code = wcode = _DTYPES[dt]
    w_ptr = b_ptr = r_ptr = z_ptr = None
    r_stride = 0
    if weight is not None:
        wcode = _norm_param(weight, "weight", index, d, dt)
        w_ptr = weight.data_ptr()
    if bias is not None:
        bcode = _norm_param(bias, "bias", index, d, dt)
        if weight is not None and bcode != wcode:
            raise TypeError("weight and bias must have one type")
        wcode, b_ptr = bcode, bias.data_ptr()
    dev = x.device
    if residual is not None:
        r_stride, r_ptr = _rows(residual, "residual", index, shape, dt), residual.data_ptr()
        z = torch.empty(shape, dtype=dt, device=dev) if z is None else _out(z, index, shape, dt, "z")
        z_ptr = z.data_ptr()
    elif z is not None:
        raise ValueError("z is written with a residual only")
    out = torch.empty(shape, dtype=dt, device=dev) if out is None else _out(out, index, shape, dt, "out")
    if stats is None:
        stats = torch.empty((2, T), dtype=torch.float32, device=dev)
    else:
        _out(stats, index, (2, T), torch.float32, "stats")
    status = lib.moe_layer_norm(x.data_ptr(), x_stride, r_ptr, r_stride, w_ptr, b_ptr, T, d, code, wcode, eps,
                                out.data_ptr(), z_ptr, stats.data_ptr(), _raw_stream(index))
    if status:
        _check(status, "moe_layer_norm")
    return (out, stats) if residual is None else (out, stats, z)


@functools.lru_cache(maxsize=256)
def moe_layer_norm_backward_workspace_bytes(T, d) -> int:
    return lib.moe_layer_norm_backward_workspace_bytes(T, d)


def moe_layer_norm_backward(dy, z, stats, weight=None, bias=True, dz=None, grads=None, workspace=None, stream=None):
    """dict(dx, dweight, dbias) for the gradient dy of moe_layer_norm's output.
    z: its z, or its x without a residual; dz: the gradient that reaches z by
    the residual path, added to dx.  dweight is None without a weight, dbias
    with bias=False.  grads: such a dict to write into."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_layer_norm_backward(dy, z, stats, weight, bias, dz, grads, workspace)
    index = _device_of(dy, "dy")
    dy_stride = _rows(dy, "dy", index)
    shape, dt, dev = dy.shape, dy.dtype, dy.device
    T, d = shape
    z_stride = _rows(z, "z", index, shape, dt)
    code = wcode = _DTYPES[dt]
    w_ptr = dz_ptr = dw_ptr = db_ptr = None
    if weight is not None:
        wcode = _norm_param(weight, "weight", index, d, dt)
        w_ptr = weight.data_ptr()
    _out(stats, index, (2, T), torch.float32, "stats")
    dz_stride = 0
    if dz is not None:
        dz_stride, dz_ptr = _rows(dz, "dz", index, shape, dt), dz.data_ptr()
    if grads is None:
        grads = dict(dx=torch.empty(shape, dtype=dt, device=dev),
                     dweight=torch.empty(d, dtype=torch.float32, device=dev) if weight is not None else None,
                     dbias=torch.empty(d, dtype=torch.float32, device=dev) if bias else None)
        dw, db = grads["dweight"], grads["dbias"]
    else:
        dw, db = grads["dweight"], grads["dbias"]
        _out(grads["dx"], index, shape, dt, "dx")
        if dw is not None:
            _out(dw, index, (d,), torch.float32, "dweight")
        if db is not None:
            _out(db, index, (d,), torch.float32, "dbias")
    if dw is not None:
        dw_ptr = dw.data_ptr()
    if db is not None:
        db_ptr = db.data_ptr()
    if workspace is None:
        size = moe_layer_norm_backward_workspace_bytes(T, d)
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    else:
        size = _workspace(workspace, index)
    status = lib.moe_layer_norm_backward(dy.data_ptr(), dy_stride, z.data_ptr(), z_stride, stats.data_ptr(), w_ptr,
                                         dz_ptr, dz_stride, T, d, code, wcode, grads["dx"].data_ptr(), dw_ptr, db_ptr,
                                         workspace.data_ptr(), size, _raw_stream(index))
    if status:
        _check(status, "moe_layer_norm_backward")
    return grads


_ROUTER_LOSS_WORKSPACE = lib.moe_router_loss_workspace_bytes()
_GRAD_NORM_WORKSPACE = lib.moe_grad_norm_workspace_bytes()


def moe_router_loss(logits, counts, balance_coef=0.01, z_coef=0.001, mask=None, accumulate=None, out=None, losses=None,
                    workspace=None, stream=None):
    """(losses [2], d_logits [T,E]) of the router's load-balancing loss and
    z-loss (both without their coefficients) and the gradient of
    balance_coef * losses[0] + z_coef * losses[1].
    counts [E] int32: the tokens each expert received, masked ones too where
    the caller routed and counted them (the mask does not change counts: for
    the balance of kept tokens alone, count their rows of topk_idx); mask [T]
    bool: tokens that the means are taken over; accumulate: a [T,E] gradient that this one is added to, in
    place (moe_backward's d_logits)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_router_loss(logits, counts, balance_coef, z_coef, mask, accumulate, out, losses, workspace)
    index = _device_of(logits, "logits")
    _contig(logits, torch.float32, "logits")
    shape, dev = logits.shape, logits.device
    T, E = shape
    _out(counts, index, (E,), torch.int32, "counts")
    m_ptr = a_ptr = None
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"mask must be bool or uint8, got {mask.dtype}")
        m_ptr = _out(mask, index, (T,), mask.dtype, "mask").data_ptr()
    if accumulate is not None:
        if out is not None:
            raise ValueError("accumulate is written in place: give it or out")
        out = _out(accumulate, index, shape, torch.float32, "accumulate")
        a_ptr = out.data_ptr()
    elif out is None:
        out = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _out(out, index, shape, torch.float32, "out")
    if losses is None:
        losses = torch.empty(2, dtype=torch.float32, device=dev)
    else:
        _out(losses, index, (2,), torch.float32, "losses")
    if workspace is None:
        size = _ROUTER_LOSS_WORKSPACE
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    else:
        size = _workspace(workspace, index)
    status = lib.moe_router_loss(logits.data_ptr(), counts.data_ptr(), m_ptr, T, E, balance_coef, z_coef, a_ptr,
                                 out.data_ptr(), losses.data_ptr(), workspace.data_ptr(), size, _raw_stream(index))
    if status:
        _check(status, "moe_router_loss")
    return losses, out


class TensorList:
    """The records of a list of tensors for moe_grad_norm and moe_adamw_step
    (made by moe_tensor_list or moe_adamw_plan), and the tensors themselves,
    so that the records' pointers stay valid."""

    def __init__(self, records, tensors, device, has_states):
        self.records, self.tensors, self.has_states = records, tensors, has_states
        self.device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.address, self.count = ctypes.addressof(records), len(records)

    def __len__(self):
        return len(self.records)


def _flat(t, name, dtypes, n, index):
    """Address of a contiguous CUDA tensor of n values (any number if None) on device `index`."""
    if t.dtype in dtypes and (n is None or t.numel() == n) and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have {n} values, got {t.numel()}")


_RECORD = struct.Struct("@7Qq3if")  # moe_adamw_tensor_t
assert _RECORD.size == ctypes.sizeof(AdamWTensor)
_F32 = (torch.float32,)
_STATES = (torch.float32, torch.uint8)


def _device_index(t):
    return t.get_device() if t.is_cuda else -2  # which no tensor's device is


def moe_tensor_list(grads) -> TensorList:
    """The list of gradients (contiguous, fp32, bf16 or fp16) for moe_grad_norm."""
    grads = list(grads)
    buf = bytearray(_RECORD.size * len(grads))
    index = _device_index(grads[0]) if grads else None
    for i, g in enumerate(grads):
        _RECORD.pack_into(buf, i * _RECORD.size, 0, 0, _flat(g, "a gradient", _DTYPES, None, index), 0, 0, 0, 0,
                          g.numel(), 0, _DTYPES[g.dtype], 0, 0.0)
    return TensorList((AdamWTensor * len(grads)).from_buffer(buf), grads, grads[0].device if grads else None, False)


def moe_adamw_state(params, bits=32):
    """Zero states for moe_adamw_plan, as a dict of its arguments m, v,
    m_scales and v_scales: fp32 values, or 8-bit codes and their scales."""
    if bits not in (32, 8):
        raise ValueError("bits must be 32 or 8")
    dt = torch.float32 if bits == 32 else torch.uint8

    def zeros():
        return [torch.zeros(p.shape, dtype=dt, device=p.device) for p in params]

    def scales():
        return [torch.ones(-(-p.numel() // 128), dtype=torch.float32, device=p.device) if bits == 8 else None
                for p in params]
    return dict(m=zeros(), v=zeros(), m_scales=scales(), v_scales=scales())


def moe_adamw_plan(params, grads, m, v, m_scales=None, v_scales=None, masters=None, decay=None) -> TensorList:
    """The list of tensors for moe_adamw_step and moe_grad_norm, made once.

    params and grads are fp32, bf16 or fp16; m and v are fp32, or uint8 codes
    with fp32 scales for every 128 values (mixed lists are fine); masters:
    fp32 masters (an entry may be None); decay: factor on the weight decay of
    each tensor (default 1).  The plan holds pointers to these tensors: make a
    new one when a tensor is replaced by another."""
    n_tensors = len(params)
    m_scales, v_scales, masters = (([None] * n_tensors) if a is None else a for a in (m_scales, v_scales, masters))
    decay = [1.0] * n_tensors if decay is None else decay
    # copies of the lists: the plan keeps the tensors, whatever the caller does with the lists
    every = tuple(tuple(a) for a in (params, grads, m, v, m_scales, v_scales, masters, decay))
    if any(len(a) != n_tensors for a in every):
        raise ValueError("the lists must have one entry for each parameter")
    buf = bytearray(_RECORD.size * n_tensors)
    index = _device_index(params[0]) if n_tensors else None
    at = 0
    for p, g, mm, vv, ms, vs, master, wd in zip(*every):
        p_ptr = _flat(p, "a parameter", _DTYPES, None, index)
        n = p.numel()
        g_ptr = _flat(g, "a gradient", _DTYPES, n, index)
        m_ptr = _flat(mm, "m", _STATES, n, index)
        v_ptr = _flat(vv, "v", (mm.dtype,), n, index)
        bits, ms_ptr, vs_ptr, master_ptr = 32, 0, 0, 0
        if mm.dtype is torch.uint8:
            if ms is None or vs is None:
                raise ValueError("8-bit states need m_scales and v_scales")
            bits = 8
            ms_ptr = _flat(ms, "m_scales", _F32, -(-n // 128), index)
            vs_ptr = _flat(vs, "v_scales", _F32, -(-n // 128), index)
        if master is not None:
            master_ptr = _flat(master, "a master", _F32, n, index)
        _RECORD.pack_into(buf, at, p_ptr, master_ptr, g_ptr, m_ptr, v_ptr, ms_ptr, vs_ptr, n, _DTYPES[p.dtype],
                          _DTYPES[g.dtype], bits, wd)
        at += _RECORD.size
    return TensorList((AdamWTensor * n_tensors).from_buffer(buf), every, params[0].device if n_tensors else None, True)


def moe_grad_norm(tensors, max_norm=float("inf"), out=None, workspace=None, stream=None):
    """[norm, factor] (fp32, on the device) over all gradients of a plan, a
    moe_tensor_list or a sequence of tensors; factor = max_norm / norm where
    the norm is larger, else 1 (NaN for a norm that is not finite): the `clip`
    argument of moe_adamw_step."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_grad_norm(tensors, max_norm, out, workspace)
    if not isinstance(tensors, TensorList):
        tensors = moe_tensor_list(tensors)
    dev = tensors.device
    index = dev.index
    _here(index, "tensors")
    if out is None:
        out = torch.empty(2, dtype=torch.float32, device=dev)
    else:
        _out(out, index, (2,), torch.float32, "out")
    if workspace is None:
        size = _GRAD_NORM_WORKSPACE
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    else:
        size = _workspace(workspace, index)
    status = lib.moe_grad_norm(tensors.address, tensors.count, max_norm, out.data_ptr(), workspace.data_ptr(), size,
                               _raw_stream(index))
    if status:
        _check(status, "moe_grad_norm")
    return out


def moe_adamw_hyper(lr, step, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1):
    """The coefficients of one step as 8 fp32 values on the host: copied into
    a device tensor, they are moe_adamw_step's `hyper` (for captured graphs)."""
    h = AdamWHyper()
    _check(lib.moe_adamw_hyper(lr, betas[0], betas[1], eps, weight_decay, step, ctypes.byref(h)), "moe_adamw_hyper")
    return torch.frombuffer(bytearray(h), dtype=torch.float32)


def moe_adamw_step(plan, lr=None, step=None, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, clip=None, hyper=None,
                   stream=None):
    """One AdamW step over the tensors of a plan, in place.  step counts from
    1; clip: moe_grad_norm's output (its second value multiplies the
    gradients; the step is skipped when that is not finite); hyper: device
    coefficients from moe_adamw_hyper, in place of lr, step, betas, eps and
    weight_decay."""
    if not plan.has_states:
        raise ValueError("moe_adamw_step needs a plan from moe_adamw_plan")
    index = plan.device.index
    if stream is not None and index != _current_device():
        with torch.cuda.stream(stream):
            return moe_adamw_step(plan, lr, step, betas, eps, weight_decay, clip, hyper)
    _here(index if stream is None else stream.device.index, "plan")
    scale = None
    if clip is not None:
        scale = _out(clip, index, (2,), torch.float32, "clip").data_ptr() + 4
    if hyper is not None:
        if lr is not None or step is not None:
            raise ValueError("give hyper, or lr and step")
        host, dev = None, _out(hyper, index, (8,), torch.float32, "hyper").data_ptr()
    else:
        if lr is None or step is None:
            raise ValueError("lr and step are needed without hyper")
        h = AdamWHyper()
        host, dev = ctypes.addressof(h), None
        status = lib.moe_adamw_hyper(lr, betas[0], betas[1], eps, weight_decay, step, host)
        if status:
            _check(status, "moe_adamw_hyper")
    status = lib.moe_adamw_step(plan.address, plan.count, host, dev, scale,
                                _raw_stream(index) if stream is None else stream.cuda_stream)
    if status:
        _check(status, "moe_adamw_step")
