"""ctypes binding of libmoe_mi355x.so (argument marshalling only).

The functions keep the C names without the ``moe_`` prefix and take torch
tensors that already live on the GPU; every step of the layer runs in the
library's HIP kernels.  Each call enqueues work on the current torch stream
(or the stream given) and returns after the launches, like the C calls.  A
non-zero status raises :class:`MoeError`.  When the library has not been
built, loading fails loudly; there is no other code path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_MI355X_LIB names another build of the same library (for example a
# second build kept for side-by-side timing); the default is the in-tree one.
LIB_PATH = os.environ.get("MOE_MI355X_LIB") or os.path.join(HERE, "_lib", "libmoe_mi355x.so")

MOE_F32, MOE_BF16 = 0, 1
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported size", -3: "workspace", -4: "HIP error"}

# Symbols declared in include/moe_mi355x.h.
EXPORTS = ("moe_route", "moe_permute", "moe_permute_workspace_size", "moe_grouped_ffn",
           "moe_grouped_ffn_workspace_size", "moe_combine", "moe_balance_stats",
           "moe_balance_stats_workspace_size", "moe_layer_forward", "moe_layer_forward_events",
           "moe_layer_forward_noalloc", "moe_workspace_size", "moe_workspace_layout",
           "moe_quantize_mxfp4", "moe_grouped_linear_mxfp4",
           "moe_grouped_linear_mxfp4_workspace_size", "moe_layer_forward_few",
           "moe_layer_forward_few_mxfp4", "moe_few_workspace_size", "moe_capacity", "moe_status_string", "moe_version")
STAGES = ("router", "topk", "dispatch", "up", "down", "combine")
# moe_version() of the interface these ctypes declarations mirror (the structs
# below must match the header's field for field)
INTERFACE_VERSION = 0x000200


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {status} ({STATUS.get(status, 'unknown')})")
        self.status = status


class Config(ctypes.Structure):
    """Mirror of moe_config."""
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int32), ("n_routed", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_shared", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("capacity_factor", ctypes.c_float),
                ("capacity", ctypes.c_int32), ("bias_mode", ctypes.c_int32),
                ("dispatch", ctypes.c_int32)]


class WsLayout(ctypes.Structure):
    """Mirror of moe_ws_layout (byte offsets into the layer workspace)."""
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("logits", "topk_idx", "topk_gate", "counts", "offsets", "n_dropped", "row_token",
                 "slot_row", "x_fp8", "x_fp8_exp", "x_fp8_wide", "total")]


class Weights(ctypes.Structure):
    """Mirror of moe_weights."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w_router", "router_bias", "w1", "b1", "w2", "b2", "ws1", "bs1", "ws2", "bs2")]


class WeightsMxfp4(ctypes.Structure):
    """Mirror of moe_weights_mxfp4."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w_router", "router_bias", "w1", "w1_scales", "b1", "w2", "w2_scales", "b2",
                 "ws1", "ws1_scales", "bs1", "ws2", "ws2_scales", "bs2")]


_LIB = None


def lib():
    """Load the library once; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing "
                               "(run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
        C = ctypes.POINTER(Config)
        sig = {
            "moe_route": (I, [C, P, P, P, P, P, P, P]),
            "moe_permute": (I, [C, P, P, P, P, P, P, P, P, P, Z, P]),
            "moe_permute_workspace_size": (Z, [C]),
            "moe_grouped_ffn": (I, [C, ctypes.c_int32, P, P, I64, P, P, P, P, P, P, P, Z, P]),
            "moe_grouped_ffn_workspace_size": (Z, [C, ctypes.c_int32, I64]),
            "moe_balance_stats": (I, [C, P, P, ctypes.c_float, P, P, P, P, Z, P]),
            "moe_balance_stats_workspace_size": (Z, [C]),
            "moe_combine": (I, [C, P, P, P, P, P, P]),
            "moe_layer_forward": (I, [C, ctypes.POINTER(Weights), P, P, P, P, P, P, Z, P]),
            "moe_layer_forward_events": (I, [C, ctypes.POINTER(Weights), P, P, P, P, P, P, Z,
                                             ctypes.POINTER(ctypes.c_void_p), P]),
            "moe_layer_forward_noalloc": (I, [C, ctypes.POINTER(Weights), P, P, P, P, P, P]),
            "moe_quantize_mxfp4": (I, [ctypes.c_int32, I64, ctypes.c_int32, P, I64, P, P, P, P]),
            "moe_grouped_linear_mxfp4": (I, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, I64,
                                             P, P, P, P, I64, P, P, P, ctypes.c_int32, P, P, Z,
                                             P]),
            "moe_grouped_linear_mxfp4_workspace_size": (Z, [ctypes.c_int32, ctypes.c_int32,
                                                            ctypes.c_int32, I64]),
            "moe_layer_forward_few": (I, [C, ctypes.POINTER(Weights), P, P, P, P, P, P, Z, P]),
            "moe_layer_forward_few_mxfp4": (I, [C, ctypes.POINTER(WeightsMxfp4), P, P, P, P, P, P,
                                                Z, P]),
            "moe_few_workspace_size": (Z, [C]),
            "moe_workspace_size": (Z, [C]),
            "moe_workspace_layout": (I, [C, ctypes.POINTER(WsLayout)]),
            "moe_capacity": (I64, [C]),
            "moe_status_string": (ctypes.c_char_p, [I]),
            "moe_version": (I, []),
        }
        # the version first: another one's calls may have other arguments
        for name in ("moe_version", *sig):
            f = getattr(L, name, None)
            if f is None:
                raise RuntimeError(f"{LIB_PATH} lacks {name}: rebuild the library")
            f.restype, f.argtypes = sig[name]
            if name == "moe_version" and f() != INTERFACE_VERSION:
                raise RuntimeError(f"{LIB_PATH} implements interface {f():#08x}, this "
                                   f"binding {INTERFACE_VERSION:#08x}: rebuild the library")
        _LIB = L
    return _LIB


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# the current stream's handle without building a Stream object (about 2.5 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(fn: str, st: int):
    if st != 0:
        raise MoeError(fn, st)


MOE_BIAS_IN_LOGIT, MOE_BIAS_SELECTION_ONLY = 0, 1
MOE_DISPATCH_BF16, MOE_DISPATCH_FP8 = 0, 1


def config(T, d_model, n_routed, top_k, n_shared, d_ff, dtype, capacity_factor=0.0,
           capacity=-1, selection_only_bias=False, dispatch_fp8=False) -> Config:
    dt = {"f32": MOE_F32, "bf16": MOE_BF16, MOE_F32: MOE_F32, MOE_BF16: MOE_BF16}[dtype]
    return Config(int(T), int(d_model), int(n_routed), int(top_k), int(n_shared), int(d_ff),
                  dt, float(capacity_factor), int(capacity),
                  MOE_BIAS_SELECTION_ONLY if selection_only_bias else MOE_BIAS_IN_LOGIT,
                  MOE_DISPATCH_FP8 if dispatch_fp8 else MOE_DISPATCH_BF16)


def capacity(cfg: Config) -> int:
    return int(lib().moe_capacity(ctypes.byref(cfg)))


def route(cfg: Config, x, w_router, router_bias, logits, topk_idx, topk_gate, stream=None):
    _check("moe_route", lib().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(w_router),
                                        _ptr(router_bias), _ptr(logits), _ptr(topk_idx),
                                        _ptr(topk_gate), _stream(stream)))


def permute_workspace_size(cfg: Config) -> int:
    return int(lib().moe_permute_workspace_size(ctypes.byref(cfg)))


def permute(cfg: Config, topk_idx, x, counts, offsets, row_token, slot_row, n_dropped,
            x_perm, ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_permute", lib().moe_permute(ctypes.byref(cfg), _ptr(topk_idx), _ptr(x),
                                            _ptr(counts), _ptr(offsets), _ptr(row_token),
                                            _ptr(slot_row), _ptr(n_dropped), _ptr(x_perm),
                                            _ptr(ws), nbytes, _stream(stream)))


def grouped_ffn_workspace_size(cfg: Config, n_groups, max_rows) -> int:
    return int(lib().moe_grouped_ffn_workspace_size(ctypes.byref(cfg), int(n_groups), int(max_rows)))


def grouped_ffn(cfg: Config, n_groups, x_rows, offsets, max_rows, w1, b1, w2, b2, h, y_rows,
                ws=None, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_grouped_ffn", lib().moe_grouped_ffn(ctypes.byref(cfg), int(n_groups), _ptr(x_rows),
                                                    _ptr(offsets), int(max_rows), _ptr(w1),
                                                    _ptr(b1), _ptr(w2), _ptr(b2), _ptr(h),
                                                    _ptr(y_rows), _ptr(ws), nbytes,
                                                    _stream(stream)))


def balance_stats_workspace_size(cfg: Config) -> int:
    return int(lib().moe_balance_stats_workspace_size(ctypes.byref(cfg)))


def balance_stats(cfg: Config, logits, topk_idx, alpha, f, P, loss, ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_balance_stats", lib().moe_balance_stats(ctypes.byref(cfg), _ptr(logits),
                                                        _ptr(topk_idx), float(alpha), _ptr(f),
                                                        _ptr(P), _ptr(loss), _ptr(ws), nbytes,
                                                        _stream(stream)))


def combine(cfg: Config, y_rows, slot_row, topk_gate, shared_out, y, stream=None):
    _check("moe_combine", lib().moe_combine(ctypes.byref(cfg), _ptr(y_rows), _ptr(slot_row),
                                            _ptr(topk_gate), _ptr(shared_out), _ptr(y),
                                            _stream(stream)))


def workspace_size(cfg: Config) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(cfg)))


def workspace_layout(cfg: Config) -> WsLayout:
    out = WsLayout()
    _check("moe_workspace_layout", lib().moe_workspace_layout(ctypes.byref(cfg), ctypes.byref(out)))
    return out


def weights(w_router, router_bias, w1, b1, w2, b2, ws1=None, bs1=None, ws2=None,
            bs2=None) -> Weights:
    return Weights(*[_ptr(t) for t in (w_router, router_bias, w1, b1, w2, b2, ws1, bs1, ws2, bs2)])


def layer_forward(cfg: Config, w: Weights, x, y, topk_idx=None, topk_gate=None, counts=None,
                  ws=None, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_layer_forward", lib().moe_layer_forward(ctypes.byref(cfg), ctypes.byref(w),
                                                        _ptr(x), _ptr(y), _ptr(topk_idx),
                                                        _ptr(topk_gate), _ptr(counts), _ptr(ws),
                                                        nbytes, _stream(stream)))


def layer_forward_noalloc(cfg: Config, w: Weights, x, y, topk_idx=None, topk_gate=None,
                          counts=None, stream=None):
    """layer_forward with the library's own static device scratch (no workspace)."""
    _check("moe_layer_forward_noalloc",
           lib().moe_layer_forward_noalloc(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), _ptr(y),
                                           _ptr(topk_idx), _ptr(topk_gate), _ptr(counts),
                                           _stream(stream)))


def layer_forward_events(cfg: Config, w: Weights, x, y, events, topk_idx=None, topk_gate=None,
                         counts=None, ws=None, stream=None):
    """layer_forward recording ``events`` (len(STAGES)+1 hipEvent_t handles) per stage."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    arr = (ctypes.c_void_p * len(events))(*events)
    _check("moe_layer_forward_events",
           lib().moe_layer_forward_events(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), _ptr(y),
                                          _ptr(topk_idx), _ptr(topk_gate), _ptr(counts), _ptr(ws),
                                          nbytes, arr, _stream(stream)))


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _on_device(*tensors):
    """The tensors given (None allowed) live on the current GPU, whose streams
    the calls use."""
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else None
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must be on the current GPU")


def quantize_mxfp4(x, codes, scales, widened=None, stream=None):
    """x [rows, d] (bf16 or f32; rows may be strided) to codes [rows, d/2] and
    scale bytes [rows, d/32] (uint8), and the values they stand for (widened
    [rows, d], x's type)."""
    _on_device(x, codes, scales, widened)
    dt = x.dtype
    _need(x.dim() == 2 and (dt is torch.bfloat16 or dt is torch.float32),
          "x must be [rows, d] bf16 or f32")
    rows, d = x.shape
    ldx, inner = x.stride()
    _need(inner == 1 or d <= 1, "elements of a row of x must be contiguous")
    _need(codes.dtype is torch.uint8 and scales.dtype is torch.uint8, "codes and scales must be uint8")
    _need(codes.shape == (rows, d // 2) and scales.shape == (rows, d // 32),
          "codes must be [rows, d/2] and scales [rows, d/32]")
    _need(widened is None or (widened.shape == (rows, d) and widened.dtype is dt),
          "widened must have x's shape and type")
    _check("moe_quantize_mxfp4", lib().moe_quantize_mxfp4(
        MOE_BF16 if dt is torch.bfloat16 else MOE_F32, rows, d, x.data_ptr(), ldx, _ptr(codes),
        _ptr(scales), _ptr(widened), _stream(stream)))


def grouped_linear_mxfp4_workspace_size(n_groups, n_out, k, max_rows) -> int:
    return int(lib().moe_grouped_linear_mxfp4_workspace_size(int(n_groups), int(n_out), int(k),
                                                             int(max_rows)))


def grouped_linear_mxfp4(x_codes, x_scales, offsets, w_codes, w_scales, y_rows, row_index=None,
                         bias=None, silu=False, ws=None, stream=None):
    """y_rows [max_rows, n_out] (bf16) of x rows [., k/2] and weights
    [n_groups, n_out, k/2]; the sizes come from the tensors."""
    _on_device(x_codes, x_scales, offsets, w_codes, w_scales, y_rows, row_index, bias, ws)
    _need(w_codes.dim() == 3 and y_rows.dim() == 2 and x_codes.dim() == 2,
          "w_codes must be [G, n_out, k/2], y_rows [rows, n_out], x_codes [., k/2]")
    u8 = torch.uint8
    _need(x_codes.dtype is u8 and x_scales.dtype is u8 and w_codes.dtype is u8 and w_scales.dtype is u8,
          "codes and scales must be uint8")
    g, n_out, kb = w_codes.shape
    max_rows, cols = y_rows.shape
    x_rows, xb = x_codes.shape
    k = 2 * kb
    _need(w_scales.shape == (g, n_out, k // 32), "w_scales must be [G, n_out, k/32]")
    _need(xb == kb and x_scales.shape == (x_rows, k // 32), "x_codes must be [., k/2], x_scales [., k/32]")
    _need(y_rows.dtype is torch.bfloat16 and cols == n_out, "y_rows must be [rows, n_out] bf16")
    _need(offsets.dtype is torch.int32 and offsets.numel() == g + 1, "offsets must be [G + 1] int32")
    if row_index is None:
        _need(x_rows >= max_rows, "x has fewer rows than y_rows (and no row_index)")
    else:
        _need(row_index.dtype is torch.int32 and row_index.numel() >= max_rows,
              "row_index must be [max_rows] int32")
    _need(bias is None or (bias.dtype is torch.bfloat16 and bias.shape == (g, n_out)),
          "bias must be [G, n_out] bf16")
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("moe_grouped_linear_mxfp4", lib().moe_grouped_linear_mxfp4(
        g, n_out, k, x_rows, _ptr(x_codes), _ptr(x_scales), _ptr(row_index), _ptr(offsets), max_rows,
        _ptr(w_codes), _ptr(w_scales), _ptr(bias), int(bool(silu)), _ptr(y_rows), _ptr(ws), nbytes,
        _stream(stream)))


def few_workspace_size(cfg: Config) -> int:
    return int(lib().moe_few_workspace_size(ctypes.byref(cfg)))


def weights_mxfp4(w_router, router_bias, w1, w1_scales, b1, w2, w2_scales, b2, ws1=None,
                  ws1_scales=None, bs1=None, ws2=None, ws2_scales=None, bs2=None) -> WeightsMxfp4:
    return WeightsMxfp4(*[_ptr(t) for t in (w_router, router_bias, w1, w1_scales, b1, w2, w2_scales,
                                            b2, ws1, ws1_scales, bs1, ws2, ws2_scales, bs2)])


def _layer_forward_few(fn: str, cfg, w, x, y, topk_idx, topk_gate, counts, ws, stream):
    _on_device(x, y, topk_idx, topk_gate, counts, ws)
    T, K = cfg.T, cfg.top_k
    act = torch.bfloat16 if cfg.dtype == MOE_BF16 else torch.float32
    _need(x.dtype is act and y.dtype is act and x.numel() == y.numel() == T * cfg.d_model,
          "x and y must be [T, d_model] of the layer's type")
    _need((topk_idx is None or (topk_idx.dtype is torch.int32 and topk_idx.numel() == T * K)) and
          (topk_gate is None or (topk_gate.dtype is torch.float32 and topk_gate.numel() == T * K)) and
          (counts is None or (counts.dtype is torch.int32 and counts.numel() == cfg.n_routed)),
          "a routing output has another size or type")
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(fn, getattr(lib(), fn)(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), _ptr(y),
                                  _ptr(topk_idx), _ptr(topk_gate), _ptr(counts), _ptr(ws), nbytes,
                                  _stream(stream)))


def layer_forward_few(cfg: Config, w: Weights, x, y, topk_idx=None, topk_gate=None, counts=None,
                      ws=None, stream=None):
    """The layer for 1 to 16 tokens (workspace: few_workspace_size)."""
    _layer_forward_few("moe_layer_forward_few", cfg, w, x, y, topk_idx, topk_gate, counts, ws, stream)


def layer_forward_few_mxfp4(cfg: Config, w: WeightsMxfp4, x, y, topk_idx=None, topk_gate=None,
                            counts=None, ws=None, stream=None):
    """layer_forward_few on MXFP4 expert weights."""
    _layer_forward_few("moe_layer_forward_few_mxfp4", cfg, w, x, y, topk_idx, topk_gate, counts, ws,
                       stream)


class HipEvents:
    """Raw HIP events (created through the HIP runtime torch already loaded)."""

    def __init__(self, n: int):
        self.rt = ctypes.CDLL("libamdhip64.so")
        self.rt.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        self.rt.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                                ctypes.c_void_p]
        self.rt.hipEventDestroy.argtypes = [ctypes.c_void_p]
        self.handles = []
        for _ in range(n):
            h = ctypes.c_void_p()
            if self.rt.hipEventCreate(ctypes.byref(h)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self.handles.append(h.value)

    def elapsed_ms(self, i: int, j: int) -> float:
        ms = ctypes.c_float()
        if self.rt.hipEventElapsedTime(ctypes.byref(ms), self.handles[i], self.handles[j]) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return float(ms.value)

    def close(self):
        for h in self.handles:
            self.rt.hipEventDestroy(h)
        self.handles = []
