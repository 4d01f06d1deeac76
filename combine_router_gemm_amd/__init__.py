"""Python binding of the MI355X MoE-layer hot path (argument marshalling only).

Every function here has the name of the C entry point it calls (include/moe.h) and only converts
torch tensors into device pointers, checks shapes and dtypes, and raises on a non-zero status. All
computation runs in the gfx950 HIP library `libmoe_gfx950.so`, built in-tree by
`python -m combine_router_gemm_amd.build`. There is no fallback: if the library is missing, every call
raises.

Tensors must be contiguous, on the current HIP device; work is enqueued on torch's current stream
unless `stream` is given.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

__all__ = ["MOE_F32", "MOE_BF16", "MOE_FP8_BLOCK", "MoeError", "Layout", "library_path", "load_library",
           "moe_route", "moe_dispatch", "moe_expert_mlp", "moe_combine", "moe_dispatch_fp8", "moe_expert_mlp_fp8",
           "moe_combine_send", "moe_combine_recv", "moe_expert_mlp_combine", "moe_dispatch_noalloc",
           "MOE_DISPATCH_NOALLOC_MAX_WORKSPACE", "MOE_W4_GROUP", "MOE_DECODE_MAX_TOKENS", "moe_w4_shapes",
           "moe_w4_codes_bytes", "moe_w4_scales_bytes", "moe_quantize_w4", "moe_dequantize_w4", "moe_expert_mlp_w4",
           "moe_expert_mlp_w4_workspace_bytes", "moe_expert_mlp_w4_tiling", "moe_layer_decode", "moe_layer_decode_w4",
           "moe_layer_decode_workspace_bytes", "moe_quantize_i8", "moe_dequantize_i8", "moe_dispatch_i8",
           "moe_expert_mlp_i8", "moe_expert_mlp_i8_workspace_bytes", "moe_expert_mlp_i8_tiling", "moe_balance_loss",
           "moe_balance_loss_workspace_bytes", "moe_combine_backward", "moe_route_backward",
           "moe_route_backward_workspace_bytes",
           "moe_expert_mlp_combine_workspace_bytes", "moe_rows_max", "moe_route_workspace_bytes", "moe_dispatch_workspace_bytes",
           "moe_expert_mlp_workspace_bytes", "moe_status_string", "EXPORTED_SYMBOLS"]

MOE_F32 = 0
MOE_BF16 = 1
MOE_FP8_BLOCK = 128  # hidden elements per fp8 block scale
MOE_DISPATCH_NOALLOC_MAX_WORKSPACE = 4 << 20  # bytes of moe_dispatch_noalloc's static scratch
MOE_W4_GROUP = 32  # consecutive k of a 4-bit weight row that share a scale
MOE_DECODE_MAX_TOKENS = 32  # tokens of moe_layer_decode / moe_layer_decode_w4

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmoe_gfx950.so"

EXPORTED_SYMBOLS = ("moe_status_string", "moe_rows_max", "moe_route_workspace_bytes", "moe_route",
                    "moe_dispatch_workspace_bytes", "moe_dispatch", "moe_expert_mlp_workspace_bytes",
                    "moe_expert_mlp", "moe_combine", "moe_dispatch_fp8", "moe_expert_mlp_fp8", "moe_combine_send",
                    "moe_combine_recv", "moe_expert_mlp_combine", "moe_expert_mlp_combine_workspace_bytes",
                    "moe_dispatch_noalloc", "moe_w4_codes_bytes", "moe_w4_scales_bytes", "moe_quantize_w4",
                    "moe_dequantize_w4", "moe_expert_mlp_w4_workspace_bytes", "moe_expert_mlp_w4_tiling",
                    "moe_expert_mlp_w4",
                    "moe_layer_decode_workspace_bytes", "moe_layer_decode", "moe_layer_decode_w4", "moe_quantize_i8",
                    "moe_dequantize_i8", "moe_dispatch_i8", "moe_expert_mlp_i8_workspace_bytes", "moe_expert_mlp_i8",
                    "moe_expert_mlp_i8_tiling", "moe_balance_loss_workspace_bytes", "moe_balance_loss", "moe_combine_backward",
                    "moe_route_backward_workspace_bytes", "moe_route_backward")


class MoeError(RuntimeError):
    """A non-zero status from the HIP library."""


class _CLayout(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("k", ctypes.c_int32), ("E", ctypes.c_int32), ("R", ctypes.c_int32),
                ("C", ctypes.c_int32), ("H", ctypes.c_int32),
                ("expert_count", ctypes.c_void_p), ("expert_kept", ctypes.c_void_p),
                ("expert_overflow", ctypes.c_void_p), ("expert_offset", ctypes.c_void_p),
                ("row_token", ctypes.c_void_p), ("row_slot", ctypes.c_void_p), ("pair_row", ctypes.c_void_p)]


_lib = None


def library_path() -> str:
    return os.path.join(_PKG, _LIB_NAME)


def load_library():
    """Load (once) and return the ctypes handle of the HIP library; raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise MoeError(f"{path} is missing: build it with `python -m combine_router_gemm_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.moe_status_string.argtypes = [i32]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_rows_max.argtypes = [i32, i32, i32, i32]
    lib.moe_rows_max.restype = i64
    lib.moe_route_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.moe_route_workspace_bytes.restype = sz
    lib.moe_route.argtypes = [vp, i32, vp, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.moe_route.restype = i32
    lib.moe_dispatch_workspace_bytes.argtypes = [i32, i32, i32]
    lib.moe_dispatch_workspace_bytes.restype = sz
    lib.moe_dispatch.argtypes = [vp, i32, vp, ctypes.POINTER(_CLayout), vp, vp, sz, vp]
    lib.moe_dispatch.restype = i32
    lib.moe_dispatch_noalloc.argtypes = [vp, i32, vp, ctypes.POINTER(_CLayout), vp, vp]
    lib.moe_dispatch_noalloc.restype = i32
    lib.moe_expert_mlp_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.moe_expert_mlp_workspace_bytes.restype = sz
    lib.moe_expert_mlp.argtypes = [vp, i32, ctypes.POINTER(_CLayout), vp, vp, i32, vp, vp, sz, vp]
    lib.moe_expert_mlp.restype = i32
    lib.moe_combine.argtypes = [vp, i32, ctypes.POINTER(_CLayout), vp, vp, vp]
    lib.moe_combine.restype = i32
    lib.moe_dispatch_fp8.argtypes = [vp, i32, vp, ctypes.POINTER(_CLayout), vp, vp, vp, sz, vp]
    lib.moe_dispatch_fp8.restype = i32
    lib.moe_expert_mlp_fp8.argtypes = [vp, vp, ctypes.POINTER(_CLayout), vp, vp, i32, vp, vp, sz, vp]
    lib.moe_expert_mlp_fp8.restype = i32
    lib.moe_expert_mlp_combine.argtypes = [vp, i32, ctypes.POINTER(_CLayout), vp, vp, i32, vp, vp, vp, vp, sz, vp]
    lib.moe_expert_mlp_combine.restype = i32
    lib.moe_expert_mlp_combine_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32]
    lib.moe_expert_mlp_combine_workspace_bytes.restype = sz
    lib.moe_combine_send.argtypes = [vp, i32, ctypes.POINTER(_CLayout), vp, vp, vp]
    lib.moe_combine_send.restype = i32
    lib.moe_combine_recv.argtypes = [vp, i32, ctypes.POINTER(_CLayout), vp, vp]
    lib.moe_combine_recv.restype = i32
    lib.moe_w4_codes_bytes.argtypes = [i64, i32]
    lib.moe_w4_codes_bytes.restype = sz
    lib.moe_w4_scales_bytes.argtypes = [i64, i32]
    lib.moe_w4_scales_bytes.restype = sz
    lib.moe_quantize_w4.argtypes = [vp, i32, i64, i32, vp, vp, vp]
    lib.moe_quantize_w4.restype = i32
    lib.moe_dequantize_w4.argtypes = [vp, vp, i64, i32, vp, i32, vp]
    lib.moe_dequantize_w4.restype = i32
    lib.moe_expert_mlp_w4_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.moe_expert_mlp_w4_workspace_bytes.restype = sz
    lib.moe_expert_mlp_w4_tiling.argtypes = [i32] * 7 + [ctypes.POINTER(ctypes.c_int)] * 2
    lib.moe_expert_mlp_w4_tiling.restype = i32
    lib.moe_expert_mlp_w4.argtypes = [vp, ctypes.POINTER(_CLayout), vp, vp, vp, vp, i32, vp, vp, sz, vp]
    lib.moe_expert_mlp_w4.restype = i32
    lib.moe_layer_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.moe_layer_decode_workspace_bytes.restype = sz
    lib.moe_layer_decode.argtypes = [vp, i32, vp, vp, i64] + [i32] * 7 + [vp] * 7 + [sz, vp]
    lib.moe_layer_decode.restype = i32
    lib.moe_layer_decode_w4.argtypes = [vp, vp, vp, i64] + [i32] * 7 + [vp] * 9 + [sz, vp]
    lib.moe_layer_decode_w4.restype = i32
    lib.moe_quantize_i8.argtypes = [vp, i32, i64, i32, vp, vp, vp]
    lib.moe_quantize_i8.restype = i32
    lib.moe_dequantize_i8.argtypes = [vp, vp, i64, i32, vp, i32, vp]
    lib.moe_dequantize_i8.restype = i32
    lib.moe_dispatch_i8.argtypes = [vp, i32, vp, ctypes.POINTER(_CLayout), vp, vp, vp, sz, vp]
    lib.moe_dispatch_i8.restype = i32
    lib.moe_expert_mlp_i8_workspace_bytes.argtypes = [i32] * 7
    lib.moe_expert_mlp_i8_workspace_bytes.restype = sz
    lib.moe_expert_mlp_i8_tiling.argtypes = [i32] * 7 + [ctypes.POINTER(ctypes.c_int)] * 3
    lib.moe_expert_mlp_i8_tiling.restype = i32
    lib.moe_expert_mlp_i8.argtypes = [vp, vp, ctypes.POINTER(_CLayout), vp, vp, vp, vp, i32, vp, vp, sz, vp]
    lib.moe_expert_mlp_i8.restype = i32
    lib.moe_balance_loss_workspace_bytes.argtypes = [i32, i32, i32]
    lib.moe_balance_loss_workspace_bytes.restype = sz
    lib.moe_balance_loss.argtypes = [vp] * 4 + [i32] * 4 + [ctypes.c_float] + [vp] * 4 + [sz, vp]
    lib.moe_balance_loss.restype = i32
    lib.moe_combine_backward.argtypes = [vp, i32, vp, ctypes.POINTER(_CLayout), vp, vp, vp, vp]
    lib.moe_combine_backward.restype = i32
    lib.moe_route_backward_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.moe_route_backward_workspace_bytes.restype = sz
    lib.moe_route_backward.argtypes = [vp, i32] + [vp] * 5 + [i32] * 4 + [vp] * 5 + [sz, vp]
    lib.moe_route_backward.restype = i32
    _lib = lib
    return lib


# ------------------------------------------------------------------------------------------------
# marshalling helpers
# ------------------------------------------------------------------------------------------------

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise MoeError(f"unsupported activation dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, shape=None, device=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise MoeError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise MoeError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise MoeError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise MoeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise MoeError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr() if t.numel() > 0 else None


def _stream_obj(stream) -> torch.cuda.Stream:
    """The torch stream object the call's kernels are enqueued on."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream))


def _stream(stream) -> Optional[int]:
    return _stream_obj(stream).cuda_stream


def _check(status: int, what: str):
    if status != 0:
        msg = load_library().moe_status_string(status).decode()
        raise MoeError(f"{what} failed: {msg} ({status})")


# ------------------------------------------------------------------------------------------------
# sizes
# ------------------------------------------------------------------------------------------------

def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def moe_rows_max(T: int, k: int, E: int, C: int) -> int:
    return int(load_library().moe_rows_max(T, k, E, C))


def moe_route_workspace_bytes(T: int, H: int, E: int, xdt: int) -> int:
    return int(load_library().moe_route_workspace_bytes(T, H, E, xdt))


def moe_dispatch_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(load_library().moe_dispatch_workspace_bytes(T, k, E))


def moe_expert_mlp_workspace_bytes(T: int, k: int, E: int, R: int, C: int, F: int, xdt: int) -> int:
    return int(load_library().moe_expert_mlp_workspace_bytes(T, k, E, R, C, F, xdt))


def moe_expert_mlp_combine_workspace_bytes(T: int, k: int, E: int, R: int, C: int, H: int, F: int, xdt: int) -> int:
    return int(load_library().moe_expert_mlp_combine_workspace_bytes(T, k, E, R, C, H, F, xdt))


def moe_w4_codes_bytes(rows: int, K: int) -> int:
    return int(load_library().moe_w4_codes_bytes(rows, K))


def moe_w4_scales_bytes(rows: int, K: int) -> int:
    return int(load_library().moe_w4_scales_bytes(rows, K))


@functools.lru_cache(maxsize=1024)
def moe_w4_shapes(*shape: int) -> tuple:
    """Shapes of the packed codes and scales (uint8) of weights [.., N, K]."""
    *lead, N, K = shape
    if N % 16 or K % MOE_W4_GROUP:
        raise MoeError(f"4-bit weights need N % 16 == 0 and K % {MOE_W4_GROUP} == 0, got [{N}, {K}]")
    return (*lead, N // 16, -(-K // 128), 1024), (*lead, N // 16, -(-K // 512), 256)


def moe_expert_mlp_w4_workspace_bytes(T: int, k: int, E: int, R: int, C: int, F: int) -> int:
    return int(load_library().moe_expert_mlp_w4_workspace_bytes(T, k, E, R, C, F))


def moe_expert_mlp_w4_tiling(T: int, k: int, E: int, R: int, C: int, H: int, F: int) -> tuple:
    """(rows per tile, parts of the down pass) that moe_expert_mlp_w4 takes for these sizes on the current device."""
    rows, parts = ctypes.c_int(), ctypes.c_int()
    st = load_library().moe_expert_mlp_w4_tiling(T, k, E, R, C, H, F, ctypes.byref(rows), ctypes.byref(parts))
    _check(st, "moe_expert_mlp_w4_tiling")
    return rows.value, parts.value


def moe_layer_decode_workspace_bytes(T: int, H: int, E: int, k: int, F: int, xdt: int) -> int:
    return int(load_library().moe_layer_decode_workspace_bytes(T, H, E, k, F, xdt))


def moe_expert_mlp_i8_workspace_bytes(T: int, k: int, E: int, R: int, C: int, H: int, F: int) -> int:
    return int(load_library().moe_expert_mlp_i8_workspace_bytes(T, k, E, R, C, H, F))


def moe_expert_mlp_i8_tiling(T: int, k: int, E: int, R: int, C: int, H: int, F: int) -> tuple:
    """(rows per tile, parts of the gate/up pass, parts of the down pass) that moe_expert_mlp_i8 takes for these sizes."""
    n = [ctypes.c_int() for _ in range(3)]
    _check(load_library().moe_expert_mlp_i8_tiling(T, k, E, R, C, H, F, *map(ctypes.byref, n)), "moe_expert_mlp_i8_tiling")
    return tuple(v.value for v in n)


def moe_balance_loss_workspace_bytes(T: int, E: int, S: int) -> int:
    return int(load_library().moe_balance_loss_workspace_bytes(T, E, S))


def moe_route_backward_workspace_bytes(T: int, H: int, E: int, xdt: int) -> int:
    return int(load_library().moe_route_backward_workspace_bytes(T, H, E, xdt))


# ------------------------------------------------------------------------------------------------
# layout descriptor
# ------------------------------------------------------------------------------------------------

class Layout:
    """The per-rank send-buffer layout: scalars plus caller-owned int32 device arrays.

    Allocates the arrays with torch on `device` (allocation is the caller's side of the ABI);
    `moe_dispatch` fills them.
    """

    def __init__(self, T: int, k: int, E: int, R: int, C: int, H: int, device="cuda"):
        self.T, self.k, self.E, self.R, self.C, self.H = T, k, E, R, C, H
        self.rows_max = max(0, min(T * k, E * C)) if (T > 0 and C > 0) else 0
        i32 = dict(dtype=torch.int32, device=device)
        self.expert_count = torch.empty(E, **i32)
        self.expert_kept = torch.empty(E, **i32)
        self.expert_overflow = torch.empty(E, **i32)
        self.expert_offset = torch.empty(E + 1, **i32)
        self.row_token = torch.empty(self.rows_max, **i32)
        self.row_slot = torch.empty(self.rows_max, **i32)
        self.pair_row = torch.empty(T, k, **i32)

    @property
    def El(self) -> int:
        return self.E // self.R

    def c_struct(self) -> _CLayout:
        def p(t):
            return t.data_ptr() if t.numel() > 0 else None
        return _CLayout(self.T, self.k, self.E, self.R, self.C, self.H,
                        p(self.expert_count), p(self.expert_kept), p(self.expert_overflow),
                        p(self.expert_offset), p(self.row_token), p(self.row_slot), p(self.pair_row))


def _workspace(nbytes: int, workspace: Optional[torch.Tensor], device, stream) -> Optional[torch.Tensor]:
    """The caller's workspace, or a temporary one. A temporary workspace is allocated on torch's current
    stream and freed when the call returns, while the kernels that use it may still be queued on
    `stream`: record_stream makes the caching allocator wait for that stream before reusing it."""
    if nbytes == 0:
        return workspace
    if workspace is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        ws.record_stream(_stream_obj(stream))
        return ws
    if _nbytes(workspace) < nbytes:
        raise MoeError(f"workspace too small: need {nbytes} bytes")
    return workspace


def _nbytes(t: Optional[torch.Tensor]) -> int:
    """Size in bytes of a workspace tensor of any element type."""
    return 0 if t is None else t.numel() * t.element_size()


# ------------------------------------------------------------------------------------------------
# the four calls
# ------------------------------------------------------------------------------------------------

def moe_route(x: torch.Tensor, w_router: torch.Tensor, logit_bias: Optional[torch.Tensor], k: int,
              logits: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
              workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Router logits, top-k ids (ties to the lower id) and softmax weights over the k selected."""
    T, H = x.shape
    E = w_router.shape[0]
    dev = x.device
    stride = 0
    if logit_bias is not None:
        if logit_bias.dim() == 1:
            _ptr(logit_bias, "logit_bias", torch.float32, (E,), dev)
        else:
            _ptr(logit_bias, "logit_bias", torch.float32, (T, E), dev)
            stride = E
    ws = _workspace(moe_route_workspace_bytes(T, H, E, _dtype_code(x)), workspace, dev, stream)
    st = load_library().moe_route(
        _ptr(x, "x", device=dev), _dtype_code(x), _ptr(w_router, "w_router", torch.float32, (E, H), dev),
        _ptr(logit_bias, "logit_bias"), stride, T, H, E, k,
        _ptr(logits, "logits", torch.float32, (T, E), dev), _ptr(topk_ids, "topk_ids", torch.int32, (T, k), dev),
        _ptr(topk_w, "topk_w", torch.float32, (T, k), dev), _ptr(ws, "workspace"),
        _nbytes(ws), _stream(stream))
    _check(st, "moe_route")


def moe_dispatch(x: torch.Tensor, topk_ids: torch.Tensor, layout: Layout, send_buf: torch.Tensor,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Histogram, capacity-clamped prefix scan and stable scatter of token rows into `send_buf`."""
    dev = x.device
    L = layout
    _ptr(x, "x", shape=(L.T, L.H), device=dev)
    _ptr(send_buf, "send_buf", x.dtype, (L.rows_max, L.H), dev)
    ws = _workspace(moe_dispatch_workspace_bytes(L.T, L.k, L.E), workspace, dev, stream)
    cl = L.c_struct()
    st = load_library().moe_dispatch(
        _ptr(x, "x"), _dtype_code(x), _ptr(topk_ids, "topk_ids", torch.int32, (L.T, L.k), dev), ctypes.byref(cl),
        _ptr(send_buf, "send_buf"), _ptr(ws, "workspace"), _nbytes(ws), _stream(stream))
    _check(st, "moe_dispatch")


def moe_dispatch_noalloc(x: torch.Tensor, topk_ids: torch.Tensor, layout: Layout, send_buf: torch.Tensor,
                         stream=None) -> None:
    """moe_dispatch with the library's static per-GPU scratch instead of a workspace (allocates nothing).
    Calls that may overlap on one GPU race; calls on one stream are ordered."""
    dev = x.device
    L = layout
    _ptr(x, "x", shape=(L.T, L.H), device=dev)
    _ptr(send_buf, "send_buf", x.dtype, (L.rows_max, L.H), dev)
    cl = L.c_struct()
    st = load_library().moe_dispatch_noalloc(
        _ptr(x, "x"), _dtype_code(x), _ptr(topk_ids, "topk_ids", torch.int32, (L.T, L.k), dev), ctypes.byref(cl),
        _ptr(send_buf, "send_buf"), _stream(stream))
    _check(st, "moe_dispatch_noalloc")


def moe_expert_mlp(send_buf: torch.Tensor, layout: Layout, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                   out_buf: torch.Tensor, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Per-expert SwiGLU MLP (grouped MFMA GEMM) on the dispatched rows; output row-aligned with send_buf."""
    dev = send_buf.device
    L = layout
    El = L.E // L.R
    F = w_gate_up.shape[1] // 2
    dt = _dtype_code(send_buf)
    _ptr(send_buf, "send_buf", shape=(L.rows_max, L.H), device=dev)
    _ptr(w_gate_up, "w_gate_up", send_buf.dtype, (El, 2 * F, L.H), dev)
    _ptr(w_down, "w_down", send_buf.dtype, (El, L.H, F), dev)
    _ptr(out_buf, "out_buf", send_buf.dtype, (L.rows_max, L.H), dev)
    ws = _workspace(moe_expert_mlp_workspace_bytes(L.T, L.k, L.E, L.R, L.C, F, dt), workspace, dev, stream)
    cl = L.c_struct()
    st = load_library().moe_expert_mlp(
        _ptr(send_buf, "send_buf"), dt, ctypes.byref(cl), _ptr(w_gate_up, "w_gate_up"), _ptr(w_down, "w_down"), F,
        _ptr(out_buf, "out_buf"), _ptr(ws, "workspace"), _nbytes(ws), _stream(stream))
    _check(st, "moe_expert_mlp")


def moe_expert_mlp_combine(send_buf: torch.Tensor, layout: Layout, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                           topk_w: torch.Tensor, out_buf: torch.Tensor, y: torch.Tensor,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_expert_mlp with moe_combine fused into its down GEMM: writes out_buf and y in one call."""
    dev = send_buf.device
    L = layout
    El = L.E // L.R
    F = w_gate_up.shape[1] // 2
    dt = _dtype_code(send_buf)
    _ptr(send_buf, "send_buf", shape=(L.rows_max, L.H), device=dev)
    _ptr(w_gate_up, "w_gate_up", send_buf.dtype, (El, 2 * F, L.H), dev)
    _ptr(w_down, "w_down", send_buf.dtype, (El, L.H, F), dev)
    _ptr(out_buf, "out_buf", send_buf.dtype, (L.rows_max, L.H), dev)
    _ptr(y, "y", send_buf.dtype, (L.T, L.H), dev)
    ws = _workspace(moe_expert_mlp_combine_workspace_bytes(L.T, L.k, L.E, L.R, L.C, L.H, F, dt), workspace, dev, stream)
    cl = L.c_struct()
    st = load_library().moe_expert_mlp_combine(
        _ptr(send_buf, "send_buf"), dt, ctypes.byref(cl), _ptr(w_gate_up, "w_gate_up"), _ptr(w_down, "w_down"), F,
        _ptr(topk_w, "topk_w", torch.float32, (L.T, L.k), dev), _ptr(out_buf, "out_buf"), _ptr(y, "y"),
        _ptr(ws, "workspace"), _nbytes(ws), _stream(stream))
    _check(st, "moe_expert_mlp_combine")


def moe_combine(out_buf: torch.Tensor, layout: Layout, topk_w: torch.Tensor, y: torch.Tensor,
                stream=None) -> None:
    """y[t] = sum of the kept slots' routing weight times their expert output row (fp32 accumulate)."""
    dev = y.device
    L = layout
    _ptr(out_buf, "out_buf", y.dtype, (L.rows_max, L.H), dev)
    _ptr(y, "y", shape=(L.T, L.H), device=dev)
    cl = L.c_struct()
    st = load_library().moe_combine(
        _ptr(out_buf, "out_buf"), _dtype_code(y), ctypes.byref(cl),
        _ptr(topk_w, "topk_w", torch.float32, (L.T, L.k), dev), _ptr(y, "y"), _stream(stream))
    _check(st, "moe_combine")


def moe_combine_send(out_buf: torch.Tensor, layout: Layout, topk_w: torch.Tensor, partial: torch.Tensor,
                     stream=None) -> None:
    """Sender-side partial rows: partial[r, t] = sum of t's kept slots on rank r of weight times expert
    output (fp32 accumulate, rounded once). partial is [R, T, H] in the activation type; slots of ranks
    holding no kept slot of t are left as they are."""
    dev = partial.device
    L = layout
    _ptr(out_buf, "out_buf", partial.dtype, (L.rows_max, L.H), dev)
    _ptr(partial, "partial", shape=(L.R, L.T, L.H), device=dev)
    cl = L.c_struct()
    st = load_library().moe_combine_send(
        _ptr(out_buf, "out_buf"), _dtype_code(partial), ctypes.byref(cl),
        _ptr(topk_w, "topk_w", torch.float32, (L.T, L.k), dev), _ptr(partial, "partial"), _stream(stream))
    _check(st, "moe_combine_send")


def moe_combine_recv(partial: torch.Tensor, layout: Layout, y: torch.Tensor, stream=None) -> None:
    """y[t] = sum over the ranks holding kept slots of t (ascending) of partial[r, t] (fp32, rounded once)."""
    dev = y.device
    L = layout
    _ptr(partial, "partial", y.dtype, (L.R, L.T, L.H), dev)
    _ptr(y, "y", shape=(L.T, L.H), device=dev)
    cl = L.c_struct()
    st = load_library().moe_combine_recv(_ptr(partial, "partial"), _dtype_code(y), ctypes.byref(cl), _ptr(y, "y"),
                                         _stream(stream))
    _check(st, "moe_combine_recv")


def moe_dispatch_fp8(x: torch.Tensor, topk_ids: torch.Tensor, layout: Layout, send_q: torch.Tensor,
                     send_scale: torch.Tensor, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_dispatch with fp8 block-scaled send rows: E4M3 codes (uint8) and one power-of-two fp32 scale
    per 128 hidden elements. x must be bf16."""
    dev = x.device
    L = layout
    _ptr(x, "x", torch.bfloat16, (L.T, L.H), dev)
    _ptr(send_q, "send_q", torch.uint8, (L.rows_max, L.H), dev)
    _ptr(send_scale, "send_scale", torch.float32, (L.rows_max, L.H // MOE_FP8_BLOCK), dev)
    ws = _workspace(moe_dispatch_workspace_bytes(L.T, L.k, L.E), workspace, dev, stream)
    cl = L.c_struct()
    st = load_library().moe_dispatch_fp8(
        _ptr(x, "x"), MOE_BF16, _ptr(topk_ids, "topk_ids", torch.int32, (L.T, L.k), dev), ctypes.byref(cl),
        _ptr(send_q, "send_q"), _ptr(send_scale, "send_scale"), _ptr(ws, "workspace"),
        _nbytes(ws), _stream(stream))
    _check(st, "moe_dispatch_fp8")


def moe_expert_mlp_fp8(send_q: torch.Tensor, send_scale: torch.Tensor, layout: Layout, w_gate_up: torch.Tensor,
                       w_down: torch.Tensor, out_buf: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """Expert SwiGLU MLP on fp8 block-scaled rows (decoded to bf16 in the GEMM); bf16 weights and output."""
    dev = send_q.device
    L = layout
    El = L.E // L.R
    F = w_gate_up.shape[1] // 2
    _ptr(send_q, "send_q", torch.uint8, (L.rows_max, L.H), dev)
    _ptr(send_scale, "send_scale", torch.float32, (L.rows_max, L.H // MOE_FP8_BLOCK), dev)
    _ptr(w_gate_up, "w_gate_up", torch.bfloat16, (El, 2 * F, L.H), dev)
    _ptr(w_down, "w_down", torch.bfloat16, (El, L.H, F), dev)
    _ptr(out_buf, "out_buf", torch.bfloat16, (L.rows_max, L.H), dev)
    ws = _workspace(moe_expert_mlp_workspace_bytes(L.T, L.k, L.E, L.R, L.C, F, MOE_BF16), workspace, dev, stream)
    cl = L.c_struct()
    st = load_library().moe_expert_mlp_fp8(
        _ptr(send_q, "send_q"), _ptr(send_scale, "send_scale"), ctypes.byref(cl), _ptr(w_gate_up, "w_gate_up"),
        _ptr(w_down, "w_down"), F, _ptr(out_buf, "out_buf"), _ptr(ws, "workspace"), _nbytes(ws),
        _stream(stream))
    _check(st, "moe_expert_mlp_fp8")


# ------------------------------------------------------------------------------------------------
# 4-bit expert weights
# ------------------------------------------------------------------------------------------------
# The calls from here on take a few microseconds on the device, as long as a handful of attribute lookups take on the
# host: their checks are one pass over the arguments, and the sizes they ask the library for are remembered by shape.

def _device(t: torch.Tensor, name: str) -> int:
    """Index of the device of a call's first tensor, which has to be the current one."""
    dev = t.get_device()
    if dev < 0:
        raise MoeError(f"{name} must be a device tensor")
    if dev != torch.cuda.current_device():
        raise MoeError(f"{name} is on device {dev}, the current one is {torch.cuda.current_device()}")
    return dev


def _arg(t: torch.Tensor, name: str, dtype, shape, dev: int) -> Optional[int]:
    """Device pointer of a contiguous tensor of this type and shape on device `dev` (None without elements)."""
    if t.dtype is not dtype:
        raise MoeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise MoeError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise MoeError(f"{name} is on {t.device}, expected device {dev}")
    if not t.is_contiguous():
        raise MoeError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


_size = functools.lru_cache(maxsize=1024)(lambda name, *args: int(getattr(load_library(), name)(*args)))


def _scratch(nbytes: int, workspace: Optional[torch.Tensor], dev: int, stream):
    """(pointer, bytes) of the caller's workspace or of a temporary one, and the tensor that holds it."""
    ws = _workspace(nbytes, workspace, dev, stream)
    if ws is None:
        return None, 0, None
    if ws.get_device() != dev or not ws.is_contiguous():
        raise MoeError(f"workspace must be a contiguous tensor on device {dev}")
    return ws.data_ptr() or None, _nbytes(ws), ws


def moe_quantize_w4(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """Weights [.., N, K] (f32 or bf16) to packed 4-bit codes and scales of the shapes moe_w4_shapes(*w.shape)."""
    cs, ss = moe_w4_shapes(*w.shape)
    dev, K = _device(w, "w"), w.shape[-1]
    st = load_library().moe_quantize_w4(
        _arg(w, "w", w.dtype, w.shape, dev), _dtype_code(w), w.numel() // K if K else 0, K,
        _arg(codes, "codes", torch.uint8, cs, dev), _arg(scales, "scales", torch.uint8, ss, dev),
        _raw_stream(stream, dev))
    if st:
        _check(st, "moe_quantize_w4")


def moe_dequantize_w4(codes: torch.Tensor, scales: torch.Tensor, w: torch.Tensor, stream=None) -> None:
    """The values packed codes and scales stand for, into w [.., N, K] (f32 or bf16, both exact)."""
    cs, ss = moe_w4_shapes(*w.shape)
    dev, K = _device(w, "w"), w.shape[-1]
    st = load_library().moe_dequantize_w4(
        _arg(codes, "codes", torch.uint8, cs, dev), _arg(scales, "scales", torch.uint8, ss, dev),
        w.numel() // K if K else 0, K, _arg(w, "w", w.dtype, w.shape, dev), _dtype_code(w), _raw_stream(stream, dev))
    if st:
        _check(st, "moe_dequantize_w4")


def _expert_shapes(El: int, F: int, H: int):
    """Packed shapes of the experts' gate/up and down weights: (codes, scales) of each."""
    return moe_w4_shapes(El, 2 * F, H) + moe_w4_shapes(El, H, F)


def moe_expert_mlp_w4(send_buf: torch.Tensor, layout: Layout, gu_codes: torch.Tensor, gu_scales: torch.Tensor,
                      dn_codes: torch.Tensor, dn_scales: torch.Tensor, out_buf: torch.Tensor,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Expert SwiGLU MLP on dispatched bf16 rows with packed 4-bit weights ([El, 2F, H] and [El, H, F])."""
    dev = _device(send_buf, "send_buf")
    L = layout
    F = gu_codes.shape[1] * 8
    gc, gs, dc, ds = _expert_shapes(L.E // L.R, F, L.H)
    u8, rows = torch.uint8, (L.rows_max, L.H)
    for name, n in (("expert_kept", L.E), ("expert_offset", L.E + 1)):  # the arrays that the kernels read
        _arg(getattr(L, name), "layout." + name, torch.int32, (n,), dev)
    need = _size("moe_expert_mlp_w4_workspace_bytes", L.T, L.k, L.E, L.R, L.C, F)
    p_ws, n_ws, ws = _scratch(need, workspace, dev, stream)
    cl = L.c_struct()
    st = load_library().moe_expert_mlp_w4(
        _arg(send_buf, "send_buf", torch.bfloat16, rows, dev), ctypes.byref(cl),
        _arg(gu_codes, "gu_codes", u8, gc, dev), _arg(gu_scales, "gu_scales", u8, gs, dev),
        _arg(dn_codes, "dn_codes", u8, dc, dev), _arg(dn_scales, "dn_scales", u8, ds, dev), F,
        _arg(out_buf, "out_buf", torch.bfloat16, rows, dev), p_ws, n_ws, _raw_stream(stream, dev))
    if st:
        _check(st, "moe_expert_mlp_w4")


# ------------------------------------------------------------------------------------------------
# the whole layer for a few tokens
# ------------------------------------------------------------------------------------------------

def _layer(name, x, w_router, logit_bias, k, R, C, F, weights, logits, topk_ids, topk_w, y, workspace, stream):
    """The call shared by moe_layer_decode and moe_layer_decode_w4: `weights` are (tensor, name, type, shape)."""
    dev, dt = _device(x, "x"), x.dtype
    T, H = x.shape
    E = w_router.shape[0]
    f32 = torch.float32
    bias, stride = None, 0
    if logit_bias is not None:
        stride = 0 if logit_bias.dim() == 1 else E
        bias = _arg(logit_bias, "logit_bias", f32, (T, E) if stride else (E,), dev)
    code = _dtype_code(x)
    p_ws, n_ws, ws = _scratch(_size("moe_layer_decode_workspace_bytes", T, H, E, k, F, code), workspace, dev, stream)
    fn = getattr(load_library(), name)
    head = (_arg(x, "x", dt, (T, H), dev),) + (() if name.endswith("w4") else (code,))
    st = fn(*head, _arg(w_router, "w_router", f32, (E, H), dev), bias, stride, T, H, E, R, k, C, F,
            *[_arg(t, n, d, s, dev) for t, n, d, s in weights],
            _arg(logits, "logits", f32, (T, E), dev), _arg(topk_ids, "topk_ids", torch.int32, (T, k), dev),
            _arg(topk_w, "topk_w", f32, (T, k), dev), _arg(y, "y", dt, (T, H), dev), p_ws, n_ws,
            _raw_stream(stream, dev))
    if st:
        _check(st, name)


def moe_layer_decode(x: torch.Tensor, w_router: torch.Tensor, logit_bias: Optional[torch.Tensor], k: int, R: int,
                     C: int, w_gate_up: torch.Tensor, w_down: torch.Tensor, logits: torch.Tensor,
                     topk_ids: torch.Tensor, topk_w: torch.Tensor, y: torch.Tensor,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """The whole layer (route, dispatch with capacity C, expert MLP, combine) for at most MOE_DECODE_MAX_TOKENS
    tokens: writes logits, topk_ids, topk_w and y."""
    H, F = x.shape[1], w_gate_up.shape[1] // 2
    El = w_router.shape[0] // R if R > 0 else 0
    weights = ((w_gate_up, "w_gate_up", x.dtype, (El, 2 * F, H)), (w_down, "w_down", x.dtype, (El, H, F)))
    _layer("moe_layer_decode", x, w_router, logit_bias, k, R, C, F, weights, logits, topk_ids, topk_w, y, workspace,
           stream)


def moe_layer_decode_w4(x: torch.Tensor, w_router: torch.Tensor, logit_bias: Optional[torch.Tensor], k: int, R: int,
                        C: int, gu_codes: torch.Tensor, gu_scales: torch.Tensor, dn_codes: torch.Tensor,
                        dn_scales: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
                        y: torch.Tensor, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_layer_decode with packed 4-bit expert weights ([El, 2F, H] and [El, H, F]) and bf16 activations."""
    if x.dtype is not torch.bfloat16:
        raise MoeError(f"x must be torch.bfloat16, got {x.dtype}")
    F, u8 = gu_codes.shape[1] * 8, torch.uint8
    gc, gs, dc, ds = _expert_shapes(w_router.shape[0] // R if R > 0 else 0, F, x.shape[1])
    weights = ((gu_codes, "gu_codes", u8, gc), (gu_scales, "gu_scales", u8, gs), (dn_codes, "dn_codes", u8, dc),
               (dn_scales, "dn_scales", u8, ds))
    _layer("moe_layer_decode_w4", x, w_router, logit_bias, k, R, C, F, weights, logits, topk_ids, topk_w, y,
           workspace, stream)


# ------------------------------------------------------------------------------------------------
# int8 experts
# ------------------------------------------------------------------------------------------------

def _opt(t: Optional[torch.Tensor], name: str, dtype, shape, dev: int) -> Optional[int]:
    """_arg of a tensor that may be left out."""
    return None if t is None else _arg(t, name, dtype, shape, dev)


def _layout(L: Layout, names, dev: int) -> _CLayout:
    """The C descriptor, after checks of the arrays that a call's kernels read or write."""
    for name in names:
        t = getattr(L, name)
        shape = ((L.E + 1,) if name == "expert_offset" else (L.T, L.k) if name == "pair_row" else
                 (L.E,) if name[0] == "e" else (L.rows_max,))
        if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
            _arg(t, "layout." + name, torch.int32, shape, dev)  # says which
    return _CLayout(L.T, L.k, L.E, L.R, L.C, L.H, L.expert_count.data_ptr() or None, L.expert_kept.data_ptr() or None,
                    L.expert_overflow.data_ptr() or None, L.expert_offset.data_ptr() or None,
                    L.row_token.data_ptr() or None, L.row_slot.data_ptr() or None, L.pair_row.data_ptr() or None)


_LAYOUT_ALL = ("expert_count", "expert_kept", "expert_overflow", "expert_offset", "row_token", "row_slot", "pair_row")


def moe_quantize_i8(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """Rows of w [.., K] (f32 or bf16) to int8 codes [.., K] and one float32 scale per row [..]."""
    dev, K = _device(w, "w"), w.shape[-1]
    st = load_library().moe_quantize_i8(
        _arg(w, "w", w.dtype, w.shape, dev), _dtype_code(w), w.numel() // K if K else 0, K,
        _arg(codes, "codes", torch.int8, w.shape, dev), _arg(scales, "scales", torch.float32, w.shape[:-1], dev),
        _raw_stream(stream, dev))
    if st:
        _check(st, "moe_quantize_i8")


def moe_dequantize_i8(codes: torch.Tensor, scales: torch.Tensor, w: torch.Tensor, stream=None) -> None:
    """code * scale into w [.., K] (f32 or bf16)."""
    dev, K = _device(w, "w"), w.shape[-1]
    st = load_library().moe_dequantize_i8(
        _arg(codes, "codes", torch.int8, w.shape, dev), _arg(scales, "scales", torch.float32, w.shape[:-1], dev),
        w.numel() // K if K else 0, K, _arg(w, "w", w.dtype, w.shape, dev), _dtype_code(w), _raw_stream(stream, dev))
    if st:
        _check(st, "moe_dequantize_i8")


def moe_dispatch_i8(x: torch.Tensor, topk_ids: torch.Tensor, layout: Layout, send_q: torch.Tensor,
                    send_scale: torch.Tensor, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """moe_dispatch with int8 send rows: codes [rows_max, H] and one float32 scale per row. x must be bf16."""
    dev = _device(x, "x")
    L = layout
    cl = _layout(L, _LAYOUT_ALL, dev)
    p_ws, n_ws, ws = _scratch(_size("moe_dispatch_workspace_bytes", L.T, L.k, L.E), workspace, dev, stream)
    st = load_library().moe_dispatch_i8(
        _arg(x, "x", torch.bfloat16, (L.T, L.H), dev), MOE_BF16, _arg(topk_ids, "topk_ids", torch.int32, (L.T, L.k), dev),
        ctypes.byref(cl), _arg(send_q, "send_q", torch.int8, (L.rows_max, L.H), dev),
        _arg(send_scale, "send_scale", torch.float32, (L.rows_max,), dev), p_ws, n_ws, _raw_stream(stream, dev))
    if st:
        _check(st, "moe_dispatch_i8")


def moe_expert_mlp_i8(send_q: torch.Tensor, send_scale: torch.Tensor, layout: Layout, gu_codes: torch.Tensor,
                      gu_scales: torch.Tensor, dn_codes: torch.Tensor, dn_scales: torch.Tensor, out_buf: torch.Tensor,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Expert SwiGLU MLP on int8 rows with int8 weights (codes [El, 2F, H] and [El, H, F], a scale per output channel);
    out_buf is bf16."""
    dev = _device(send_q, "send_q")
    L = layout
    El, F = L.E // L.R, gu_codes.shape[1] // 2
    i8, f32 = torch.int8, torch.float32
    cl = _layout(L, ("expert_kept", "expert_offset"), dev)
    need = _size("moe_expert_mlp_i8_workspace_bytes", L.T, L.k, L.E, L.R, L.C, L.H, F)
    p_ws, n_ws, ws = _scratch(need, workspace, dev, stream)
    st = load_library().moe_expert_mlp_i8(
        _arg(send_q, "send_q", i8, (L.rows_max, L.H), dev), _arg(send_scale, "send_scale", f32, (L.rows_max,), dev),
        ctypes.byref(cl), _arg(gu_codes, "gu_codes", i8, (El, 2 * F, L.H), dev),
        _arg(gu_scales, "gu_scales", f32, (El, 2 * F), dev), _arg(dn_codes, "dn_codes", i8, (El, L.H, F), dev),
        _arg(dn_scales, "dn_scales", f32, (El, L.H), dev), F,
        _arg(out_buf, "out_buf", torch.bfloat16, (L.rows_max, L.H), dev), p_ws, n_ws, _raw_stream(stream, dev))
    if st:
        _check(st, "moe_expert_mlp_i8")


# ------------------------------------------------------------------------------------------------
# training the router
# ------------------------------------------------------------------------------------------------

def moe_balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, weight: float, loss: torch.Tensor,
                     expert_count: torch.Tensor, d_logits: Optional[torch.Tensor] = None,
                     seq_offset: Optional[torch.Tensor] = None, token_mask: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Per-expert counts [S, E], balance loss [1] and its gradient [T, E] over S sequences (seq_offset [S + 1]; one of all
    tokens without it). token_mask [T] is uint8 or bool, 0 for tokens that do not count."""
    dev = _device(logits, "logits")
    T, E = logits.shape
    k = topk_ids.shape[1]
    S = 1 if seq_offset is None else seq_offset.shape[0] - 1
    f32, i32 = torch.float32, torch.int32
    mask_t = torch.bool if token_mask is not None and token_mask.dtype is torch.bool else torch.uint8
    p_ws, n_ws, ws = _scratch(_size("moe_balance_loss_workspace_bytes", T, E, S), workspace, dev, stream)
    st = load_library().moe_balance_loss(
        _arg(logits, "logits", f32, (T, E), dev), _arg(topk_ids, "topk_ids", i32, (T, k), dev),
        _opt(seq_offset, "seq_offset", i32, (S + 1,), dev), _opt(token_mask, "token_mask", mask_t, (T,), dev), T, E, k, S,
        weight, _arg(loss, "loss", f32, (1,), dev), _arg(expert_count, "expert_count", i32, (S, E), dev),
        _opt(d_logits, "d_logits", f32, (T, E), dev), p_ws, n_ws, _raw_stream(stream, dev))
    if st:
        _check(st, "moe_balance_loss")


def moe_combine_backward(dy: torch.Tensor, out_buf: torch.Tensor, layout: Layout, topk_w: torch.Tensor,
                         d_topk_w: torch.Tensor, d_out_buf: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of moe_combine: d_topk_w [T, k], and d_out_buf [rows_max, H] unless it is left out."""
    dev = _device(dy, "dy")
    L, f32 = layout, torch.float32
    cl = _layout(L, ("pair_row",), dev)
    st = load_library().moe_combine_backward(
        _arg(dy, "dy", dy.dtype, (L.T, L.H), dev), _dtype_code(dy),
        _arg(out_buf, "out_buf", dy.dtype, (L.rows_max, L.H), dev), ctypes.byref(cl),
        _arg(topk_w, "topk_w", f32, (L.T, L.k), dev), _arg(d_topk_w, "d_topk_w", f32, (L.T, L.k), dev),
        _opt(d_out_buf, "d_out_buf", dy.dtype, (L.rows_max, L.H), dev), _raw_stream(stream, dev))
    if st:
        _check(st, "moe_combine_backward")


def moe_route_backward(x: torch.Tensor, w_router: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
                       d_topk_w: Optional[torch.Tensor], d_logits_in: Optional[torch.Tensor], d_logits: torch.Tensor,
                       d_x: Optional[torch.Tensor] = None, d_w_router: Optional[torch.Tensor] = None,
                       d_bias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """Gradients of moe_route from those of the routing weights (d_topk_w) and of the logits (d_logits_in), either of which
    may be None: d_logits [T, E], and d_x [T, H], d_w_router [E, H], d_bias [E] unless they are left out."""
    dev, dt = _device(x, "x"), x.dtype
    T, H = x.shape
    E, k = w_router.shape[0], topk_ids.shape[1]
    f32 = torch.float32
    code = _dtype_code(x)
    p_ws, n_ws, ws = _scratch(_size("moe_route_backward_workspace_bytes", T, H, E, code), workspace, dev, stream)
    st = load_library().moe_route_backward(
        _arg(x, "x", dt, (T, H), dev), code, _arg(w_router, "w_router", f32, (E, H), dev),
        _arg(topk_ids, "topk_ids", torch.int32, (T, k), dev), _arg(topk_w, "topk_w", f32, (T, k), dev),
        _opt(d_topk_w, "d_topk_w", f32, (T, k), dev), _opt(d_logits_in, "d_logits_in", f32, (T, E), dev), T, H, E, k,
        _arg(d_logits, "d_logits", f32, (T, E), dev), _opt(d_x, "d_x", dt, (T, H), dev),
        _opt(d_w_router, "d_w_router", f32, (E, H), dev), _opt(d_bias, "d_bias", f32, (E,), dev), p_ws, n_ws,
        _raw_stream(stream, dev))
    if st:
        _check(st, "moe_route_backward")
