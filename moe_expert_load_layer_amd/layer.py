"""Python calls of the operators around the balancer: the gate, the experts' 8-bit
grouped products, the layer for a few tokens and AdamW (contracts in
include/ep_balance.h).  As in the package's other calls, torch supplies memory and the
current stream, arguments are checked here, and outputs may be given or are allocated.
"""
from __future__ import annotations

import ctypes
from typing import List, Optional, Sequence

import numpy as np
import torch

from . import (EPBalanceError, Layout, _check, _CLayout, _held, ep_dispatch_layout, ep_load_histogram, ep_plan_quota,
               ep_replica_grad_reduce, ep_slot_fill, lib)
from . import _arg as _arg_or_raise

EP_DTYPE_F32, EP_DTYPE_BF16, EP_DTYPE_FP8 = 0, 1, 2
EP_MAX_FEW_TOKENS = 64

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_FLOATS = {torch.float32: EP_DTYPE_F32, torch.bfloat16: EP_DTYPE_BF16}
_FP8 = torch.float8_e4m3fn


class _CGate(ctypes.Structure):
    _fields_ = [("num_experts", _i32), ("top_k", _i32), ("num_groups", _i32), ("topk_groups", _i32),
                ("logits_dtype", _i32), ("scale", ctypes.c_float), ("bias", _vp)]


class _CMatrix(ctypes.Structure):
    _fields_ = [("data", _vp), ("scale", _vp), ("stride", _i64), ("scale_stride", _i64)]


class _CMatmul(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_scale", _vp), ("x_rows", _i64), ("rows", _vp), ("rows_div", _i32), ("groups", _i32),
                ("offsets", _vp), ("m", _i64), ("n", _i64), ("k", _i64), ("w", _CMatrix), ("slot_w", _CMatrix),
                ("layout", ctypes.POINTER(_CLayout)), ("y", _vp)]


class _CWgrad(ctypes.Structure):
    _fields_ = [("dy", _vp), ("x", _vp), ("dy_stride", _i64), ("x_stride", _i64), ("m", _i64), ("n", _i64),
                ("k", _i64), ("groups", _i32), ("offsets", _vp), ("layout", ctypes.POINTER(_CLayout)), ("out", _vp),
                ("slot_out", _vp), ("out_stride", _i64), ("slot_out_stride", _i64)]


class _CSwiglu(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_scale", _vp), ("x_rows", _i64), ("rows", _vp), ("rows_div", _i32), ("groups", _i32),
                ("offsets", _vp), ("m", _i64), ("inter", _i64), ("k", _i64), ("gate", _CMatrix), ("up", _CMatrix),
                ("slot_gate", _CMatrix), ("slot_up", _CMatrix), ("layout", ctypes.POINTER(_CLayout)), ("weights", _vp),
                ("weights_count", _i64), ("h", _vp), ("h_scale", _vp), ("keep_dtype", _i32), ("keep", _vp), ("keep_scale", _vp),
                ("sums8", _i32)]


class _CSwigluBackward(ctypes.Structure):
    _fields_ = [("dy", _vp), ("dy_scale", _vp), ("dy_rows", _i64), ("rows", _vp), ("rows_div", _i32), ("groups", _i32),
                ("offsets", _vp), ("m", _i64), ("inter", _i64), ("k", _i64), ("down", _CMatrix), ("slot_down", _CMatrix),
                ("layout", ctypes.POINTER(_CLayout)), ("weights", _vp), ("weights_count", _i64), ("keep_dtype", _i32),
                ("keep", _vp), ("keep_scale", _vp), ("grad", _vp), ("q", _vp), ("q_scale", _vp), ("grad_weights", _vp),
                ("grad_weights_dtype", _i32), ("pos", _vp), ("pairs", _i64), ("ws", _vp), ("ws_bytes", _sz),
                ("sums8", _i32)]


class _CWgradMixed(ctypes.Structure):
    _fields_ = [("dy", _vp), ("dy_rows", _i64), ("dy_stride", _i64), ("x", _vp), ("x_scale", _vp), ("x_rows", _i64),
                ("dy_places", _vp), ("x_places", _vp), ("rows_div", _i32), ("groups", _i32), ("offsets", _vp),
                ("m", _i64), ("n", _i64), ("k", _i64), ("layout", ctypes.POINTER(_CLayout)), ("out", _vp),
                ("slot_out", _vp), ("out_stride", _i64), ("slot_out_stride", _i64), ("ws", _vp), ("ws_bytes", _sz)]


class _CExperts(ctypes.Structure):
    _fields_ = [("hidden", _i32), ("inter", _i32), ("dtype", _i32), ("gate", _CMatrix), ("up", _CMatrix),
                ("down", _CMatrix)]


class _CAdamW(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", _i64), ("seed", ctypes.c_uint32), ("state_bits", _i32), ("grad_dtype", _i32)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the library's entry points, called once when it is loaded."""
    p = ctypes.POINTER
    L.ep_gate_topk.argtypes = [_vp, _i64, _i64, p(_CGate), _vp, _vp, _vp]
    L.ep_gate_topk_backward.argtypes = [_vp, _vp, _vp, _i64, p(_CGate), _vp, _vp]
    L.ep_scale_stride.argtypes = [_i64]
    L.ep_scale_stride.restype = _i64
    L.ep_quant_rows.argtypes = [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp]
    L.ep_swiglu_quant.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp]
    L.ep_quant_blocks.argtypes = [_vp, _i32, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp]
    L.ep_grouped_matmul.argtypes = [p(_CMatmul), _vp]
    L.ep_grouped_wgrad.argtypes = [p(_CWgrad), _vp]
    L.ep_grouped_wgrad_mixed.argtypes = [p(_CWgradMixed), _vp]
    L.ep_wgrad_mixed_workspace_bytes.argtypes = [_i64, _i64]
    L.ep_wgrad_mixed_workspace_bytes.restype = _sz
    L.ep_grouped_swiglu.argtypes = [p(_CSwiglu), _vp]
    L.ep_swiglu_backward_workspace_bytes.argtypes = [_i64, _i64]
    L.ep_swiglu_backward_workspace_bytes.restype = _sz
    L.ep_grouped_swiglu_backward.argtypes = [p(_CSwigluBackward), _vp]
    L.ep_moe_combine.argtypes = [_vp, _i64, _vp, _vp, _i64, _i32, _i64, _vp, _vp]
    L.ep_few_tokens_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32]
    L.ep_few_tokens_workspace_bytes.restype = _sz
    L.ep_moe_few_tokens.argtypes = [_vp, _i64, _i32, _vp, _i64, p(_CGate), p(_CExperts), _vp, _i64, _vp, _vp, _vp,
                                    _sz, _vp]
    L.ep_adamw_step.argtypes = [_vp, _i32, p(_CAdamW), _vp]
    L.ep_adamw_values.argtypes = [_vp, _i32, _vp, _vp, _vp]
    for f in ("ep_gate_topk", "ep_gate_topk_backward", "ep_quant_rows", "ep_swiglu_quant", "ep_quant_blocks",
              "ep_grouped_matmul", "ep_grouped_wgrad", "ep_grouped_wgrad_mixed", "ep_grouped_swiglu",
              "ep_grouped_swiglu_backward", "ep_moe_combine", "ep_moe_few_tokens", "ep_adamw_step", "ep_adamw_values"):
        getattr(L, f).restype = ctypes.c_int


# These calls are a few microseconds of GPU time each in decoding, so that the checks and the stream's lookup take
# the cheapest forms: one chain of comparisons where all is well, the messages only where it is not.

def _arg(t: Optional[torch.Tensor], dtype: torch.dtype, shape, name: str) -> torch.Tensor:
    """A contiguous device tensor of exactly this dtype and shape."""
    if t is not None and t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t
    return _arg_or_raise(t, dtype, shape, name)


def _ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    """The given stream, or torch's current one, as a pointer."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else stream.cuda_stream


def _rows(t: torch.Tensor, dtypes, name: str) -> int:
    """A device matrix whose rows are contiguous; returns its row stride."""
    if t.is_cuda and t.dtype in dtypes and t.dim() == 2:
        (m, n), (sm, sn) = t.shape, t.stride()
        if m > 1 and sm >= n and (sn == 1 or n <= 1):
            return sm
    if not t.is_cuda:
        raise EPBalanceError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise EPBalanceError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 2:
        raise EPBalanceError(f"{name} must have two dimensions, got shape {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise EPBalanceError(f"{name} must have contiguous rows")
    if t.shape[0] <= 1:
        return t.shape[1]
    if t.stride(0) < t.shape[1]:
        raise EPBalanceError(f"{name} must have rows that do not overlap")
    return t.stride(0)


def _out(t: Optional[torch.Tensor], dtype: torch.dtype, shape, device, name: str, stream) -> torch.Tensor:
    if t is None:
        return _held(torch.empty(shape, dtype=dtype, device=device), stream)
    return _arg(t, dtype, shape, name)


def _gate(num_experts: int, k: int, bias, num_groups: int, topk_groups: int, scale: float, dtype) -> _CGate:
    if bias is not None:
        _arg(bias, torch.float32, (num_experts,), "bias")
    return _CGate(num_experts, k, num_groups, topk_groups, _FLOATS[dtype], scale,
                  None if bias is None else bias.data_ptr())


def ep_gate_topk(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None, num_groups: int = 1,
                 topk_groups: int = 1, scale: float = 1.0, ids=None, weights=None, stream=None):
    """logits fp32 or bf16 [T][E] -> (ids int32 [T][k], weights float32 [T][k])."""
    stride = _rows(logits, (torch.float32, torch.bfloat16), "logits")
    T, E = logits.shape
    ids = _out(ids, torch.int32, (T, k), logits.device, "ids", stream)
    weights = _out(weights, torch.float32, (T, k), logits.device, "weights", stream)
    g = _gate(E, k, bias, num_groups, topk_groups, scale, logits.dtype)
    rc = lib().ep_gate_topk(_ptr(logits), stride, T, ctypes.byref(g), _ptr(ids), _ptr(weights), _stream(stream))
    _check(rc, "ep_gate_topk")
    return ids, weights


def ep_gate_topk_backward(ids: torch.Tensor, weights: torch.Tensor, grad_weights: torch.Tensor, num_experts: int,
                          scale: float = 1.0, dtype=torch.float32, grad_logits=None, stream=None) -> torch.Tensor:
    """The gradient of ep_gate_topk's weights -> grad_logits [T][E] in `dtype`."""
    if dtype not in _FLOATS:
        raise EPBalanceError(f"grad_logits must be float32 or bfloat16, got {dtype}")
    if ids.dim() != 2:
        raise EPBalanceError(f"ids must be [tokens][k], got shape {tuple(ids.shape)}")
    T, k = ids.shape
    _arg(ids, torch.int32, (T, k), "ids")
    _arg(weights, torch.float32, (T, k), "weights")
    _arg(grad_weights, torch.float32, (T, k), "grad_weights")
    grad_logits = _out(grad_logits, dtype, (T, num_experts), ids.device, "grad_logits", stream)
    g = _gate(num_experts, k, None, 1, 1, scale, dtype)
    rc = lib().ep_gate_topk_backward(_ptr(ids), _ptr(weights), _ptr(grad_weights), T, ctypes.byref(g),
                                     _ptr(grad_logits), _stream(stream))
    _check(rc, "ep_gate_topk_backward")
    return grad_logits


def ep_scale_stride(cols: int) -> int:
    """Scale bytes of a row of `cols` values: its blocks of 128, up to a multiple of 4."""
    return (cols + 511) // 512 * 4 if cols > 0 else 0


def _up128(n: int) -> int:
    return (n + 127) // 128 * 128


def ep_quant_rows(x: torch.Tensor, q=None, scale=None, stream=None):
    """x fp32 or bf16 [M][K] -> (q float8_e4m3fn [M][K up to 128], scale uint8 [M][ep_scale_stride(K)])."""
    stride = _rows(x, (torch.float32, torch.bfloat16), "x")
    M, K = x.shape
    q = _out(q, _FP8, (M, _up128(K)), x.device, "q", stream)
    scale = _out(scale, torch.uint8, (M, ep_scale_stride(K)), x.device, "scale", stream)
    _check(lib().ep_quant_rows(_ptr(x), _FLOATS[x.dtype], M, K, stride, _ptr(q), _ptr(scale), _stream(stream)),
           "ep_quant_rows")
    return q, scale


def ep_swiglu_quant(gate_up: torch.Tensor, q=None, scale=None, stream=None):
    """silu(g) * u of bf16 rows [M][2 I] (g, then u), as ep_quant_rows gives it."""
    if gate_up.dim() != 2 or gate_up.shape[1] % 2:
        raise EPBalanceError(f"gate_up must be [rows][2 * inter], got shape {tuple(gate_up.shape)}")
    M, I = gate_up.shape[0], gate_up.shape[1] // 2
    _arg(gate_up, torch.bfloat16, (M, 2 * I), "gate_up")
    q = _out(q, _FP8, (M, _up128(I)), gate_up.device, "q", stream)
    scale = _out(scale, torch.uint8, (M, ep_scale_stride(I)), gate_up.device, "scale", stream)
    _check(lib().ep_swiglu_quant(_ptr(gate_up), M, I, _ptr(q), _ptr(scale), _stream(stream)), "ep_swiglu_quant")
    return q, scale


def ep_quant_blocks(w: torch.Tensor, transpose: bool = False, q=None, scale=None, stream=None):
    """w fp32 or bf16 [G][N][K] -> (q float8_e4m3fn [G][N][K up to 128], scale uint8 [G][blocks of N][blocks of K]);
    transpose: of the transposed matrices, [G][K][N up to 128] and [G][blocks of K][blocks of N]."""
    if w.dim() != 3 or w.dtype not in _FLOATS or not w.is_cuda:
        raise EPBalanceError("w must be a device tensor [groups][rows][cols] in float32 or bfloat16")
    G, N, K = w.shape
    if G and not w[0].is_contiguous():
        raise EPBalanceError("w must have contiguous matrices")
    a, b = (K, N) if transpose else (N, K)
    q = _out(q, _FP8, (G, a, _up128(b)), w.device, "q", stream)
    scale = _out(scale, torch.uint8, (G, _up128(a) // 128, _up128(b) // 128), w.device, "scale", stream)
    rc = lib().ep_quant_blocks(_ptr(w), _FLOATS[w.dtype], G, w.stride(0), N, K, int(transpose), _ptr(q), _ptr(scale),
                               _stream(stream))
    _check(rc, "ep_quant_blocks")
    return q, scale


def _matrix(data: torch.Tensor, scale: Optional[torch.Tensor], rows: int, cols: int, name: str) -> _CMatrix:
    """[experts][rows][cols] (bf16) or [experts][rows][cols up to 128] with scales (8 bits); experts may be apart."""
    fp8 = scale is not None
    shape, stride = data.shape, data.stride()
    if fp8:
        blocks, width = (rows + 127) // 128, (cols + 127) // 128 * 128
        if (data.is_cuda and data.dtype is _FP8 and len(shape) == 3 and shape[1] == rows and shape[2] == width and
                stride[2] == 1 and stride[1] == width and scale.is_cuda and scale.dtype is torch.uint8 and
                scale.shape == (shape[0], blocks, width // 128)):
            ss = scale.stride()
            if (ss[2] == 1 or width == 128) and (ss[1] == width // 128 or blocks == 1):
                return _CMatrix(data.data_ptr(), scale.data_ptr(), stride[0], ss[0])
    elif (data.is_cuda and data.dtype is torch.bfloat16 and len(shape) == 3 and shape[1] == rows and
          shape[2] == cols and stride[2] == 1 and stride[1] == cols):
        return _CMatrix(data.data_ptr(), None, stride[0] * 2, 0)
    if not data.is_cuda or data.dim() != 3 or data.dtype != (_FP8 if fp8 else torch.bfloat16):
        raise EPBalanceError(f"{name} must be a device tensor [experts][rows][cols] in "
                             f"{'float8_e4m3fn' if fp8 else 'bfloat16'}, got {data.dtype} {tuple(data.shape)}")
    width = _up128(cols) if fp8 else cols
    if tuple(data.shape[1:]) != (rows, width):
        raise EPBalanceError(f"{name} must have shape [experts][{rows}][{width}], got {tuple(data.shape)}")
    if data.stride(2) != 1 and width > 1 or data.stride(1) != width and rows > 1:
        raise EPBalanceError(f"{name} must have contiguous matrices")
    m = _CMatrix(data.data_ptr(), None, data.stride(0) * data.element_size(), 0)
    if fp8:
        shape = (data.shape[0], _up128(rows) // 128, width // 128)
        if not scale.is_cuda or scale.dtype != torch.uint8 or tuple(scale.shape) != shape:
            raise EPBalanceError(f"{name}'s scale must be a uint8 device tensor of shape {shape}")
        if scale.shape[0] and not scale[0].is_contiguous():
            raise EPBalanceError(f"{name}'s scale must have contiguous matrices")
        m.scale, m.scale_stride = scale.data_ptr(), scale.stride(0)
    return m


def _groups(offsets: Optional[torch.Tensor], layout: Optional[Layout], count: int) -> int:
    if layout is not None:
        if count != layout.num_experts:
            raise EPBalanceError(f"with a layout there is one matrix for each of its {layout.num_experts} experts")
        count = layout.num_phys
    if offsets is not None:
        _arg(offsets, torch.int32, (count + 1,), "offsets")
    elif count != 1:
        raise EPBalanceError("offsets are required with more than one group")
    return count


def ep_grouped_matmul(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                      offsets: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None, rows_div: int = 1,
                      layout: Optional[Layout] = None, slot_w=None, slot_w_scale=None, y=None,
                      stream=None) -> torch.Tensor:
    """y[i] = w_g x[r(i)] in bf16 for the rows i of group g, offsets[g] .. offsets[g + 1] - 1.

    x, x_scale from ep_quant_rows, w [G][N][K up to 128] and w_scale from ep_quant_blocks.  rows int32 [M]:
    r(i) = rows[i] // rows_div (negative: a row of zeros).  layout: the groups are its physical slots, w the native
    experts' matrices and slot_w, slot_w_scale the spare slots'."""
    if x.dim() != 2 or w.dim() != 3 or x.shape[1] % 128 or x.shape[1] != w.shape[2]:
        raise EPBalanceError(f"x [rows][k] and w [groups][n][k] must share k, a multiple of 128: got {tuple(x.shape)} "
                             f"and {tuple(w.shape)}")
    K, N = x.shape[1], w.shape[1]
    _arg(x, _FP8, x.shape, "x")
    _arg(x_scale, torch.uint8, (x.shape[0], ep_scale_stride(K)), "x_scale")
    G = _groups(offsets, layout, w.shape[0])
    X = M = x.shape[0]
    if rows is not None:
        if rows.dim() != 1:
            raise EPBalanceError("rows must be [output rows]")
        _arg(rows, torch.int32, rows.shape, "rows")
        M = rows.shape[0]
    y = _out(y, torch.bfloat16, (M, N), x.device, "y", stream)
    p = _CMatmul(x.data_ptr(), x_scale.data_ptr(), X, None if rows is None else rows.data_ptr(), rows_div, G,
                 None if offsets is None else offsets.data_ptr(), M, N, K, _matrix(w, w_scale, N, K, "w"), _CMatrix(),
                 None, y.data_ptr())
    if layout is not None:
        p.layout = ctypes.pointer(layout.c)
        if layout.num_spare:
            if slot_w is None or slot_w_scale is None or slot_w.shape[0] != layout.num_spare:
                raise EPBalanceError(f"slot_w and slot_w_scale must hold the layout's {layout.num_spare} spare slots")
            p.slot_w = _matrix(slot_w, slot_w_scale, N, K, "slot_w")
    _check(lib().ep_grouped_matmul(ctypes.byref(p), _stream(stream)), "ep_grouped_matmul")
    return y


def _gradient(t: Optional[torch.Tensor], shape, device, name: str, stream) -> torch.Tensor:
    """float32 [matrices][N][K], the matrices contiguous but perhaps apart."""
    if t is None:
        return _held(torch.empty(shape, dtype=torch.float32, device=device), stream)
    if not t.is_cuda or t.dtype != torch.float32 or tuple(t.shape) != shape:
        raise EPBalanceError(f"{name} must be a float32 device tensor of shape {shape}")
    if shape[0] and not t[0].is_contiguous():
        raise EPBalanceError(f"{name} must have contiguous matrices")
    return t


def ep_grouped_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                     layout: Optional[Layout] = None, out=None, slot_out=None, stream=None):
    """sum over the rows i of group g of dy[i][n] x[i][k] -> float32 [G][N][K]; dy, x bf16.

    With a layout the groups are its physical slots: returns (native [E][N][K], spare [S][N][K]), the gradients that
    ep_replica_grad_reduce folds.  out, slot_out may have rows of more than N * K values (packed expert rows)."""
    ds, xs = _rows(dy, (torch.bfloat16,), "dy"), _rows(x, (torch.bfloat16,), "x")
    if dy.shape[0] != x.shape[0]:
        raise EPBalanceError(f"dy and x must have the same rows, got {dy.shape[0]} and {x.shape[0]}")
    M, N, K = dy.shape[0], dy.shape[1], x.shape[1]
    if offsets is not None and (offsets.dim() != 1 or offsets.shape[0] < 2):
        raise EPBalanceError("offsets must be [groups + 1]")
    G = _groups(offsets, layout, layout.num_experts if layout is not None else
                1 if offsets is None else offsets.shape[0] - 1)

    shape = (layout.num_experts if layout is not None else G, N, K)
    out = _gradient(out, shape, dy.device, "out", stream)
    p = _CWgrad(dy.data_ptr(), x.data_ptr(), ds, xs, M, N, K, G, None if offsets is None else offsets.data_ptr(),
                None, out.data_ptr(), None, out.stride(0), 0)
    if layout is not None:
        p.layout = ctypes.pointer(layout.c)
        slot_out = _gradient(slot_out, (layout.num_spare, N, K), dy.device, "slot_out", stream)
        if layout.num_spare:
            p.slot_out, p.slot_out_stride = slot_out.data_ptr(), slot_out.stride(0)
    _check(lib().ep_grouped_wgrad(ctypes.byref(p), _stream(stream)), "ep_grouped_wgrad")
    return out if layout is None else (out, slot_out)


def _places(t: Optional[torch.Tensor], name: str) -> int:
    """The length of a list of places, int32 [rows]."""
    if t.dim() != 1:
        raise EPBalanceError(f"{name} must be [output rows]")
    _arg(t, torch.int32, t.shape, name)
    return t.shape[0]


def _workspace(ws: Optional[torch.Tensor], need: int, device, stream) -> torch.Tensor:
    """The workspace that is given, or a new one; the caller holds it until its call, or another output takes its place."""
    if ws is None:
        ws = _held(torch.empty(max(16, need), dtype=torch.uint8, device=device), stream)
    elif not (ws.is_cuda and ws.is_contiguous()):
        raise EPBalanceError("ws must be a contiguous device tensor")
    return ws


def ep_wgrad_mixed_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().ep_wgrad_mixed_workspace_bytes(int(rows), int(cols)))


def ep_grouped_wgrad_mixed(dy: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor,
                           offsets: Optional[torch.Tensor] = None, cols: Optional[int] = None, dy_rows=None,
                           x_rows=None, rows_div: int = 1, layout: Optional[Layout] = None, out=None, slot_out=None,
                           ws=None, stream=None):
    """ep_grouped_wgrad with x in 8 bits: sum over the rows i of group g of dy[d(i)][n] x[r(i)][k] -> float32 [G][N][cols].

    x, x_scale as ep_quant_rows or ep_grouped_swiglu wrote rows of `cols` values (default: all that x has).
    d(i) = dy_rows[i] // rows_div, r(i) = x_rows[i] // rows_div (int32 [M]; None: i; both: the same list; negative or
    too large: the row adds nothing).  With a layout: (native, spare), as ep_grouped_wgrad.
    ws: ep_wgrad_mixed_workspace_bytes(rows of x, cols) bytes."""
    ds = _rows(dy, (torch.bfloat16,), "dy")
    if x.dim() != 2 or x.shape[1] % 128:
        raise EPBalanceError(f"x must be [rows][columns up to a multiple of 128], got shape {tuple(x.shape)}")
    K, N = x.shape[1] if cols is None else cols, dy.shape[1]
    if K < 1 or _up128(K) != x.shape[1]:
        raise EPBalanceError(f"cols must be the columns that x's {x.shape[1]} hold, got {cols}")
    _arg(x, _FP8, x.shape, "x")
    _arg(x_scale, torch.uint8, (x.shape[0], ep_scale_stride(K)), "x_scale")
    lengths = {name: t.shape[0] if places is None else _places(places, name + "_rows")
               for name, t, places in (("dy", dy, dy_rows), ("x", x, x_rows))}
    M = lengths["dy"]
    if lengths["x"] != M:
        raise EPBalanceError(f"dy and x must give the same rows, got {M} and {lengths['x']}")
    if dy_rows is not None and x_rows is not None and dy_rows.data_ptr() != x_rows.data_ptr():
        raise EPBalanceError("dy_rows and x_rows must be one list where both are given")
    if offsets is not None and (offsets.dim() != 1 or offsets.shape[0] < 2):
        raise EPBalanceError("offsets must be [groups + 1]")
    G = _groups(offsets, layout, layout.num_experts if layout is not None else
                1 if offsets is None else offsets.shape[0] - 1)
    shape = (layout.num_experts if layout is not None else G, N, K)
    out = _gradient(out, shape, dy.device, "out", stream)
    p = _CWgradMixed(dy.data_ptr(), dy.shape[0], ds, x.data_ptr(), x_scale.data_ptr(), x.shape[0],
                     None if dy_rows is None else dy_rows.data_ptr(), None if x_rows is None else x_rows.data_ptr(),
                     rows_div, G, None if offsets is None else offsets.data_ptr(), M, N, K, None, out.data_ptr(), None,
                     out.stride(0), 0)
    ws = _workspace(ws, ep_wgrad_mixed_workspace_bytes(x.shape[0], K), dy.device, stream)
    p.ws, p.ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    if layout is not None:
        p.layout = ctypes.pointer(layout.c)
        slot_out = _gradient(slot_out, (layout.num_spare, N, K), dy.device, "slot_out", stream)
        if layout.num_spare:
            p.slot_out, p.slot_out_stride = slot_out.data_ptr(), slot_out.stride(0)
    _check(lib().ep_grouped_wgrad_mixed(ctypes.byref(p), _stream(stream)), "ep_grouped_wgrad_mixed")
    return out if layout is None else (out, slot_out)


def _slot_matrix(layout: Layout, data, scale, rows: int, cols: int, name: str) -> _CMatrix:
    if data is None or scale is None or data.shape[0] != layout.num_spare:
        raise EPBalanceError(f"{name} and its scale must hold the layout's {layout.num_spare} spare slots")
    return _matrix(data, scale, rows, cols, name)


def _pair_weights(weights: torch.Tensor, count: Optional[int]) -> int:
    """The length of float32 weights, one for each pair; count: what it has to be."""
    if weights.dim() != 1:
        raise EPBalanceError(f"weights must be [pairs], got shape {tuple(weights.shape)}")
    _arg(weights, torch.float32, weights.shape if count is None else (count,), "weights")
    return weights.shape[0]


def ep_grouped_swiglu(x: torch.Tensor, x_scale: torch.Tensor, gate: torch.Tensor, gate_scale: torch.Tensor,
                      up: torch.Tensor, up_scale: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                      rows: Optional[torch.Tensor] = None, rows_div: int = 1, weights: Optional[torch.Tensor] = None,
                      keep: Optional[torch.dtype] = None, layout: Optional[Layout] = None, slot_gate=None,
                      slot_gate_scale=None, slot_up=None, slot_up_scale=None, h=None, h_scale=None, kept=None,
                      kept_scale=None, stream=None, sums8: bool = False):
    """h[i] = w_i silu(gate_g x[r(i)]) * (up_g x[r(i)]) in 8 bits, for the rows i of group g, in one product.

    x, x_scale from ep_quant_rows, gate and up [G][I][K up to 128] with the scales of ep_quant_blocks; offsets, rows,
    rows_div and layout as for ep_grouped_matmul.  weights float32, one for each pair that rows may name (a pair past
    them has no input; without rows: [M]); None: 1.  keep: None, or the type in which the two products are kept for
    ep_grouped_swiglu_backward, torch.bfloat16 ([M][2 I]) or torch.float8_e4m3fn ([M][2 * (I up to 128)] and scales).
    sums8: the 8-bit instruction's sums, as ep_grouped_matmul has them, in place of fp32's: little more than half the
    time for many rows, but one value in 300 is rounded to 8 bits the other way.
    Returns (h, h_scale, kept, kept_scale), the last two None where there are none."""
    if x.dim() != 2 or gate.dim() != 3 or x.shape[1] % 128 or x.shape[1] != gate.shape[2]:
        raise EPBalanceError(f"x [rows][k] and gate [groups][inter][k] must share k, a multiple of 128: got "
                             f"{tuple(x.shape)} and {tuple(gate.shape)}")
    X, K, I = x.shape[0], x.shape[1], gate.shape[1]
    _arg(x, _FP8, x.shape, "x")
    _arg(x_scale, torch.uint8, (X, ep_scale_stride(K)), "x_scale")
    if up.shape != gate.shape:
        raise EPBalanceError(f"gate and up must have one shape, got {tuple(gate.shape)} and {tuple(up.shape)}")
    if gate_scale is None or up_scale is None:
        raise EPBalanceError("gate_scale and up_scale are required")
    G = _groups(offsets, layout, gate.shape[0])
    M = X if rows is None else _places(rows, "rows")
    count = 0 if weights is None else _pair_weights(weights, None if rows is not None else M)
    h = _out(h, _FP8, (M, _up128(I)), x.device, "h", stream)
    h_scale = _out(h_scale, torch.uint8, (M, ep_scale_stride(I)), x.device, "h_scale", stream)
    if keep is None:
        if kept is not None or kept_scale is not None:
            raise EPBalanceError("kept needs keep, its type")
    elif keep is torch.bfloat16:
        kept = _out(kept, keep, (M, 2 * I), x.device, "kept", stream)
        kept_scale = None
    elif keep is _FP8:
        kept = _out(kept, keep, (M, 2 * _up128(I)), x.device, "kept", stream)
        kept_scale = _out(kept_scale, torch.uint8, (M, ep_scale_stride(2 * _up128(I))), x.device, "kept_scale", stream)
    else:
        raise EPBalanceError(f"keep must be None, torch.bfloat16 or torch.float8_e4m3fn, got {keep}")
    p = _CSwiglu(x.data_ptr(), x_scale.data_ptr(), X, None if rows is None else rows.data_ptr(), rows_div, G,
                 None if offsets is None else offsets.data_ptr(), M, I, K, _matrix(gate, gate_scale, I, K, "gate"),
                 _matrix(up, up_scale, I, K, "up"), _CMatrix(), _CMatrix(), None,
                 None if weights is None else weights.data_ptr(), count, h.data_ptr(), h_scale.data_ptr(),
                 EP_DTYPE_FP8 if keep is _FP8 else EP_DTYPE_BF16, None if kept is None else kept.data_ptr(),
                 None if kept_scale is None else kept_scale.data_ptr(), int(bool(sums8)))
    if layout is not None:
        p.layout = ctypes.pointer(layout.c)
        if layout.num_spare:
            p.slot_gate = _slot_matrix(layout, slot_gate, slot_gate_scale, I, K, "slot_gate")
            p.slot_up = _slot_matrix(layout, slot_up, slot_up_scale, I, K, "slot_up")
    _check(lib().ep_grouped_swiglu(ctypes.byref(p), _stream(stream)), "ep_grouped_swiglu")
    return h, h_scale, kept, kept_scale


def ep_swiglu_backward_workspace_bytes(rows: int, inter: int) -> int:
    return int(lib().ep_swiglu_backward_workspace_bytes(int(rows), int(inter)))


def ep_grouped_swiglu_backward(dy: torch.Tensor, dy_scale: torch.Tensor, down: torch.Tensor, down_scale: torch.Tensor,
                               kept: torch.Tensor, kept_scale: Optional[torch.Tensor] = None,
                               offsets: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                               rows_div: int = 1, weights: Optional[torch.Tensor] = None,
                               pos: Optional[torch.Tensor] = None, weights_dtype: torch.dtype = torch.float32,
                               layout: Optional[Layout] = None, slot_down=None, slot_down_scale=None, grad=None, q=None,
                               q_scale=None, grad_weights=None, ws=None, stream=None, sums8: bool = False):
    """The gradient of ep_grouped_swiglu, from the gradient of the block's output and what was kept.

    dy, dy_scale: the output's gradient, a row for each token, from ep_quant_rows; down [G][I][columns of dy] and its
    scales from ep_quant_blocks(transpose=True); kept, kept_scale, weights, offsets, rows, rows_div, layout as there.
    Returns (grad bf16 [M][2 I], the dy of the projections' weight gradient; q and q_scale, the same in 8 bits
    [M][2 * (I up to 128)], the x of the grouped product that gives the input gradient; grad_weights).  grad_weights,
    where weights are given: in weights_dtype, float32 or bfloat16, by pair where pos (int32, each pair's position)
    is given, else by position.  sums8: as there."""
    if dy.dim() != 2 or down.dim() != 3 or dy.shape[1] % 128 or dy.shape[1] != down.shape[2]:
        raise EPBalanceError(f"dy [rows][k] and down [groups][inter][k] must share k, a multiple of 128: got "
                             f"{tuple(dy.shape)} and {tuple(down.shape)}")
    X, K, I = dy.shape[0], dy.shape[1], down.shape[1]
    _arg(dy, _FP8, dy.shape, "dy")
    _arg(dy_scale, torch.uint8, (X, ep_scale_stride(K)), "dy_scale")
    if down_scale is None:
        raise EPBalanceError("down_scale is required")
    if weights_dtype not in _FLOATS:
        raise EPBalanceError(f"weights_dtype must be float32 or bfloat16, got {weights_dtype}")
    G = _groups(offsets, layout, down.shape[0])
    M = X if rows is None else _places(rows, "rows")
    wide = 2 * _up128(I)
    fp8 = kept_scale is not None
    _arg(kept, _FP8 if fp8 else torch.bfloat16, (M, wide if fp8 else 2 * I), "kept")
    if fp8:
        _arg(kept_scale, torch.uint8, (M, ep_scale_stride(wide)), "kept_scale")
    grad = _out(grad, torch.bfloat16, (M, 2 * I), dy.device, "grad", stream)
    q = _out(q, _FP8, (M, wide), dy.device, "q", stream)
    q_scale = _out(q_scale, torch.uint8, (M, ep_scale_stride(wide)), dy.device, "q_scale", stream)
    p = _CSwigluBackward(dy.data_ptr(), dy_scale.data_ptr(), X, None if rows is None else rows.data_ptr(), rows_div, G,
                         None if offsets is None else offsets.data_ptr(), M, I, K,
                         _matrix(down, down_scale, I, K, "down"), _CMatrix(), None, None, 0,
                         EP_DTYPE_FP8 if fp8 else EP_DTYPE_BF16, kept.data_ptr(),
                         kept_scale.data_ptr() if fp8 else None, grad.data_ptr(), q.data_ptr(), q_scale.data_ptr())
    p.sums8 = int(bool(sums8))
    if weights is not None:
        p.weights_count = _pair_weights(weights, None if rows is not None else M)
        pairs = M if pos is None else _places(pos, "pos")
        grad_weights = _out(grad_weights, weights_dtype, (pairs,), dy.device, "grad_weights", stream)
        p.weights, p.grad_weights, p.grad_weights_dtype = weights.data_ptr(), grad_weights.data_ptr(), _FLOATS[weights_dtype]
        p.pos, p.pairs = None if pos is None else pos.data_ptr(), pairs
        ws = _workspace(ws, ep_swiglu_backward_workspace_bytes(M, I), dy.device, stream)
        p.ws, p.ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    elif pos is not None or grad_weights is not None:
        raise EPBalanceError("grad_weights and pos need weights")
    if layout is not None:
        p.layout = ctypes.pointer(layout.c)
        if layout.num_spare:
            p.slot_down = _slot_matrix(layout, slot_down, slot_down_scale, I, K, "slot_down")
    _check(lib().ep_grouped_swiglu_backward(ctypes.byref(p), _stream(stream)), "ep_grouped_swiglu_backward")
    return grad, q, q_scale, grad_weights


def ep_moe_combine(y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t][j] y[pos[t][j]]; y bf16 [rows][H], pos int32 [T][k], weights float32 [T][k]."""
    if y.dim() != 2 or pos.dim() != 2:
        raise EPBalanceError("y must be [rows][hidden] and pos [tokens][k]")
    _arg(y, torch.bfloat16, y.shape, "y")
    _arg(pos, torch.int32, pos.shape, "pos")
    _arg(weights, torch.float32, pos.shape, "weights")
    (T, k), H = pos.shape, y.shape[1]
    out = _out(out, torch.bfloat16, (T, H), y.device, "out", stream)
    _check(lib().ep_moe_combine(_ptr(y), y.shape[0], _ptr(pos), _ptr(weights), T, k, H, _ptr(out), _stream(stream)),
           "ep_moe_combine")
    return out


def ep_few_tokens_workspace_bytes(num_tokens: int, top_k: int, hidden: int, inter: int) -> int:
    return int(lib().ep_few_tokens_workspace_bytes(int(num_tokens), int(top_k), int(hidden), int(inter)))


def ep_moe_few_tokens(x: torch.Tensor, logits: torch.Tensor, k: int, gate: torch.Tensor, up: torch.Tensor,
                      down: torch.Tensor, gate_scale=None, up_scale=None, down_scale=None, bias=None,
                      num_groups: int = 1, topk_groups: int = 1, scale: float = 1.0, out=None, ids=None, weights=None,
                      ws=None, stream=None):
    """The whole layer for at most EP_MAX_FEW_TOKENS tokens -> (out bf16 [T][H], ids int32 [T][k], weights [T][k]).

    x bf16 [T][H], logits [T][E] as for ep_gate_topk, gate and up [E][I][H], down [E][H][I] in bf16 or, with the
    scales of ep_quant_blocks, in 8 bits.  ws: ep_few_tokens_workspace_bytes(T, k, H, I) bytes."""
    xs = _rows(x, (torch.bfloat16,), "x")
    ls = _rows(logits, (torch.float32, torch.bfloat16), "logits")
    (T, H), E = x.shape, logits.shape[1]
    if logits.shape[0] != T:
        raise EPBalanceError(f"x and logits must have the same tokens, got {T} and {logits.shape[0]}")
    if T > EP_MAX_FEW_TOKENS:
        raise EPBalanceError(f"at most {EP_MAX_FEW_TOKENS} tokens, got {T}")
    scales = (gate_scale, up_scale, down_scale)
    if any(s is None for s in scales) and any(s is not None for s in scales):
        raise EPBalanceError("gate_scale, up_scale and down_scale go together")
    I = gate.shape[1] if gate.dim() == 3 else 0
    for t, name in ((gate, "gate"), (up, "up"), (down, "down")):
        if t.dim() != 3 or t.shape[0] != E:
            raise EPBalanceError(f"{name} must hold the {E} experts of the logits, got shape {tuple(t.shape)}")
    e = _CExperts(H, I, EP_DTYPE_BF16 if gate_scale is None else EP_DTYPE_FP8, _matrix(gate, gate_scale, I, H, "gate"),
                  _matrix(up, up_scale, I, H, "up"), _matrix(down, down_scale, H, I, "down"))
    out = _out(out, torch.bfloat16, (T, H), x.device, "out", stream)
    ids = _out(ids, torch.int32, (T, k), x.device, "ids", stream)
    weights = _out(weights, torch.float32, (T, k), x.device, "weights", stream)
    g = _gate(E, k, bias, num_groups, topk_groups, scale, logits.dtype)
    if ws is None:
        ws = _held(torch.empty(max(16, ep_few_tokens_workspace_bytes(T, k, H, I)), dtype=torch.uint8,
                               device=x.device), stream)
    elif not (ws.is_cuda and ws.is_contiguous()):
        raise EPBalanceError("ws must be a contiguous device tensor")
    rc = lib().ep_moe_few_tokens(_ptr(x), xs, T, _ptr(logits), ls, ctypes.byref(g), ctypes.byref(e), _ptr(out), H,
                                 _ptr(ids), _ptr(weights), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "ep_moe_few_tokens")
    return out, ids, weights


class ExpertRows:
    """8-bit weights of a layer's experts, one packed row of bytes each: gate above up [2 I][H], down [H][I], then
    their scales.  A row is what ep_slot_fill copies, so a buffer of spare slots has the same views.

    gate, up, gate_scale, up_scale are the halves of gate_up, which ep_grouped_swiglu and ep_moe_few_tokens take.  One
    scale byte may cover rows of both where inter is no multiple of 128: then they are None, unless the rows are made
    with apart=True, which gives either its own scales and leaves gate_up None."""

    def __init__(self, count: int, hidden: int, inter: int, device, apart: bool = False):
        self.hidden, self.inter = hidden, inter
        hp, ip, hb, ib = _up128(hidden), _up128(inter), _up128(hidden) // 128, _up128(inter) // 128
        self._halves = apart or inter % 128 == 0
        nb = 2 * ib if self._halves else _up128(2 * inter) // 128
        ends = np.cumsum([2 * inter * hp, hidden * ip, nb * hb, hb * ib])
        self.rows = torch.zeros((count, int(-(-ends[3] // 16) * 16)), dtype=torch.uint8, device=device)
        part = lambda a, b, n, k: self.rows[:, a:b].unflatten(1, (n, k))     # noqa: E731
        self.gate_up = part(0, ends[0], 2 * inter, hp).view(_FP8)
        self.down = part(ends[0], ends[1], hidden, ip).view(_FP8)
        self.gate_up_scale, self.down_scale = part(ends[1], ends[2], nb, hb), part(ends[2], ends[3], hb, ib)
        self.gate = self.up = self.gate_scale = self.up_scale = None
        if self._halves:
            self.gate, self.up = self.gate_up[:, :inter], self.gate_up[:, inter:]
            self.gate_scale, self.up_scale = self.gate_up_scale[:, :ib], self.gate_up_scale[:, ib:]
        if inter % 128 and apart:
            self.gate_up = self.gate_up_scale = None

    def load(self, gate_up: torch.Tensor, down: torch.Tensor) -> "ExpertRows":
        """Rounds fp32 or bf16 matrices [E][2 I][H] and [E][H][I] into the rows."""
        if self.gate_up is None:
            parts = [(gate_up[:, :self.inter], self.gate, self.gate_scale),
                     (gate_up[:, self.inter:], self.up, self.up_scale)]
        else:
            parts = [(gate_up, self.gate_up, self.gate_up_scale)]
        for w, q, s in parts + [(down, self.down, self.down_scale)]:
            wq, ws = ep_quant_blocks(w)
            q.view(torch.uint8).copy_(wq.view(torch.uint8))
            s.copy_(ws)
        return self


class ExpertBackwardRows:
    """The same experts' matrices transposed, as a backward pass takes them: down_t [I][H up to 128], both_t [H][2 * (I up
    to 128)] (gate's transpose beside up's, each up to whole blocks) and their scales, packed rows as ExpertRows'."""

    def __init__(self, count: int, hidden: int, inter: int, device):
        self.hidden, self.inter = hidden, inter
        hp, ip, hb, ib = _up128(hidden), _up128(inter), _up128(hidden) // 128, _up128(inter) // 128
        ends = np.cumsum([hidden * 2 * ip, inter * hp, hb * 2 * ib, ib * hb])
        self.rows = torch.zeros((count, int(-(-ends[3] // 16) * 16)), dtype=torch.uint8, device=device)
        part = lambda a, b, n, k: self.rows[:, a:b].unflatten(1, (n, k))     # noqa: E731
        self.both_t = part(0, ends[0], hidden, 2 * ip).view(_FP8)
        self.down_t = part(ends[0], ends[1], inter, hp).view(_FP8)
        self.both_t_scale, self.down_t_scale = part(ends[1], ends[2], hb, 2 * ib), part(ends[2], ends[3], ib, hb)

    def load(self, gate_up: torch.Tensor, down: torch.Tensor) -> "ExpertBackwardRows":
        """Rounds the matrices that ExpertRows.load takes."""
        I, ip, ib = self.inter, _up128(self.inter), _up128(self.inter) // 128
        for w, q, s in ((gate_up[:, :I], self.both_t[:, :, :ip], self.both_t_scale[:, :, :ib]),
                        (gate_up[:, I:], self.both_t[:, :, ip:], self.both_t_scale[:, :, ib:]),
                        (down, self.down_t, self.down_t_scale)):
            wq, ws = ep_quant_blocks(w, transpose=True)
            q.view(torch.uint8).copy_(wq.view(torch.uint8))
            s.copy_(ws)
        return self


def _route(logits, k, layout, experts, slots, bias, num_groups, topk_groups, scale):
    """The balanced path of one layer: gate, load, plan, dispatch order, replicas into the spare slots."""
    ids, weights = ep_gate_topk(logits, k, bias, num_groups, topk_groups, scale)
    pairs = ids.view(1, -1)
    load, ws, status = ep_load_histogram(pairs, layout)
    plan = ep_plan_quota(load, layout, status=status)
    offsets, pos, src = ep_dispatch_layout(pairs, layout, plan.phy_quota, plan.log2phy, plan.logcnt, ws)
    if layout.num_spare:
        ep_slot_fill(experts.rows, plan.phy2log[0], layout, slots.rows)
    return ids, weights, plan, status, offsets, pos, src


def run_layer(x: torch.Tensor, logits: torch.Tensor, k: int, layout: Layout, experts: ExpertRows, slots: ExpertRows,
              bias=None, num_groups: int = 1, topk_groups: int = 1, scale: float = 1.0):
    """One balanced mixture-of-experts layer over the tokens of all ranks, on the current stream: gate, load, plan,
    replicas into the spare slots, dispatch order, the experts' products over the physical slots, combine.

    x bf16 [tokens][H], logits [tokens][E] (rank by rank, the same number of tokens each); experts: the native
    experts' rows, slots: the spare slots' (filled here).  Returns a dict: out bf16 [tokens][H], ids, weights, plan,
    offsets, pos, src, h (the 8-bit input of the second product and its scales)."""
    if x.dim() != 2 or logits.dim() != 2 or x.shape[0] != logits.shape[0]:
        raise EPBalanceError(f"x [tokens][hidden] and logits [tokens][experts] must have the same tokens, got "
                             f"{tuple(x.shape)} and {tuple(logits.shape)}")
    if experts.gate_up is None:
        raise EPBalanceError("experts made apart with inter no multiple of 128 have no gate_up")
    ids, weights, plan, status, offsets, pos, src = _route(logits, k, layout, experts, slots, bias, num_groups,
                                                           topk_groups, scale)
    spare = (slots.gate_up, slots.gate_up_scale, slots.down, slots.down_scale) if layout.num_spare else (None,) * 4
    xq, xs = ep_quant_rows(x)
    up = ep_grouped_matmul(xq, xs, experts.gate_up, experts.gate_up_scale, offsets[0], rows=src[0], rows_div=k,
                           layout=layout, slot_w=spare[0], slot_w_scale=spare[1])
    h = ep_swiglu_quant(up)
    y = ep_grouped_matmul(*h, experts.down, experts.down_scale, offsets[0], layout=layout, slot_w=spare[2],
                          slot_w_scale=spare[3])
    out = ep_moe_combine(y, pos.view(-1, k), weights)
    return dict(out=out, ids=ids, weights=weights, plan=plan, status=status, offsets=offsets[0], pos=pos[0],
                src=src[0], up=up, h=h, y=y)


def run_layer_train(x: torch.Tensor, logits: torch.Tensor, k: int, layout: Layout, experts: ExpertRows,
                    slots: ExpertRows, bias=None, num_groups: int = 1, topk_groups: int = 1, scale: float = 1.0,
                    keep: torch.dtype = _FP8, sums8: bool = False):
    """run_layer's layer in a training step: returns a dict with out bf16 [tokens][H], ids, weights, plan, status,
    offsets, pos, src, and what run_layer_backward needs besides.

    What is kept of the activations for it: x and the weighted silu(g) u in 8 bits, as the products take them, and g
    and u in `keep` (torch.float8_e4m3fn or torch.bfloat16).  experts and slots need gate and up with their own scales
    (ExpertRows).  sums8: as in ep_grouped_swiglu, here and in the backward pass."""
    if x.dim() != 2 or logits.dim() != 2 or x.shape[0] != logits.shape[0]:
        raise EPBalanceError(f"x [tokens][hidden] and logits [tokens][experts] must have the same tokens, got "
                             f"{tuple(x.shape)} and {tuple(logits.shape)}")
    if experts.gate is None or (layout.num_spare and slots.gate is None):
        raise EPBalanceError("experts and slots need gate and up with their own scales: inter a multiple of 128, or "
                             "ExpertRows(apart=True)")
    if keep not in (_FP8, torch.bfloat16):
        raise EPBalanceError(f"keep must be torch.float8_e4m3fn or torch.bfloat16, got {keep}")
    ids, weights, plan, status, offsets, pos, src = _route(logits, k, layout, experts, slots, bias, num_groups,
                                                           topk_groups, scale)
    spare = layout.num_spare > 0
    xq, xs = ep_quant_rows(x)
    h, hs, kept, ks = ep_grouped_swiglu(
        xq, xs, experts.gate, experts.gate_scale, experts.up, experts.up_scale, offsets[0], rows=src[0], rows_div=k,
        weights=weights.view(-1), keep=keep, layout=layout, slot_gate=slots.gate if spare else None,
        slot_gate_scale=slots.gate_scale if spare else None, slot_up=slots.up if spare else None,
        slot_up_scale=slots.up_scale if spare else None, sums8=sums8)
    y = ep_grouped_matmul(h, hs, experts.down, experts.down_scale, offsets[0], layout=layout,
                          slot_w=slots.down if spare else None, slot_w_scale=slots.down_scale if spare else None)
    out = ep_moe_combine(y, pos.view(-1, k), torch.ones_like(weights))
    return dict(out=out, ids=ids, weights=weights, plan=plan, status=status, offsets=offsets[0], pos=pos[0], src=src[0],
                x=(xq, xs), h=(h, hs), kept=(kept, ks), top_k=k, scale=scale, logits_dtype=logits.dtype,
                hidden=x.shape[1], inter=experts.inter, sums8=sums8)


def run_layer_backward(kept: dict, grad_out: torch.Tensor, layout: Layout, experts: ExpertBackwardRows,
                       slots: ExpertBackwardRows):
    """The gradients of run_layer_train's layer, from what it returned and grad_out, bf16 [tokens][H].

    Returns a dict: x bf16 [tokens][H], logits [tokens][E] in the logits' type, gate_up float32 [E][2 I][H], down
    float32 [E][H][I], the replicas' shares folded into their experts'.  Roundings to 8 bits count as the identity.
    experts: the native experts' transposed matrices, slots: the spare slots' (filled here)."""
    k, H, I = kept["top_k"], kept["hidden"], kept["inter"]
    ids, weights, plan, offsets, pos, src = (kept[n] for n in ("ids", "weights", "plan", "offsets", "pos", "src"))
    _arg(grad_out, torch.bfloat16, (ids.shape[0], H), "grad_out")
    if (experts.hidden, experts.inter) != (H, I):
        raise EPBalanceError(f"experts must be of hidden {H} and inter {I}, got {experts.hidden} and {experts.inter}")
    spare = layout.num_spare > 0
    if spare and H * I % 4:
        raise EPBalanceError(f"with spare slots hidden * inter must be a multiple of 4, got {H} * {I}")
    if spare:
        ep_slot_fill(experts.rows, plan.phy2log[0], layout, slots.rows)
    dq, ds = ep_quant_rows(grad_out)
    grad, q, qs, dw = ep_grouped_swiglu_backward(
        dq, ds, experts.down_t, experts.down_t_scale, *kept["kept"], offsets, rows=src, rows_div=k,
        weights=weights.view(-1), pos=pos, layout=layout, slot_down=slots.down_t if spare else None,
        slot_down_scale=slots.down_t_scale if spare else None, sums8=kept["sums8"])
    dx = ep_grouped_matmul(q, qs, experts.both_t, experts.both_t_scale, offsets, layout=layout,
                           slot_w=slots.both_t if spare else None,
                           slot_w_scale=slots.both_t_scale if spare else None)
    out = dict(x=ep_moe_combine(dx, pos.view(-1, k), torch.ones_like(weights)),
               logits=ep_gate_topk_backward(ids, weights, dw.view(-1, k), layout.num_experts, kept["scale"],
                                            kept["logits_dtype"]))
    for name, dy, dy_rows, (xq, xs), x_rows, cols in (("gate_up", grad, None, kept["x"], src, H),
                                                      ("down", grad_out, src, kept["h"], None, I)):
        native, replicas = ep_grouped_wgrad_mixed(dy, xq, xs, offsets, cols=cols, dy_rows=dy_rows, x_rows=x_rows,
                                                  rows_div=k, layout=layout)
        if spare:
            ep_replica_grad_reduce(native.flatten(1), replicas.flatten(1), plan.log2phy[0], plan.logcnt[0], layout)
        out[name] = native
    return out


class AdamW:
    """AdamW over a list of fp32 tensors, updated in place by one launch a step.

    bits: 32 or 8, the width of the two moments (8: blocks of 128 with a scale byte, rounded stochastically from
    `seed`, repeatable).  copies: bf16 tensors that receive the new parameters, or None.  Keeps the parameters, their
    moments (exp_avg, exp_avg_sq and, with 8 bits, their *_scale lists) and `step_count`."""

    def __init__(self, params: Sequence[torch.Tensor], bits: int = 32, copies: Optional[Sequence[torch.Tensor]] = None,
                 lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.01, seed: int = 0):
        if bits not in (8, 32):
            raise EPBalanceError(f"bits must be 8 or 32, got {bits}")
        self.params, self.bits = list(params), bits
        for i, p in enumerate(self.params):
            _arg(p, torch.float32, p.shape, f"params[{i}]")
        self.copies = None if copies is None else list(copies)
        if self.copies is not None:
            if len(self.copies) != len(self.params):
                raise EPBalanceError("copies must be one for each parameter")
            for i, (c, p) in enumerate(zip(self.copies, self.params)):
                _arg(c, torch.bfloat16, p.shape, f"copies[{i}]")
        self.lr, self.beta1, self.beta2, self.eps, self.weight_decay = lr, beta1, beta2, eps, weight_decay
        self.seed, self.step_count = int(seed) & 0xFFFFFFFF, 0
        state = torch.float32 if bits == 32 else torch.uint8
        self.exp_avg = [torch.zeros(p.shape, dtype=state, device=p.device) for p in self.params]
        self.exp_avg_sq = [torch.zeros(p.shape, dtype=state, device=p.device) for p in self.params]
        self.exp_avg_scale: Optional[List[torch.Tensor]] = None
        self.exp_avg_sq_scale: Optional[List[torch.Tensor]] = None
        if bits == 8:
            self.exp_avg_scale, self.exp_avg_sq_scale = (
                [torch.ones((p.numel() + 127) // 128, dtype=torch.uint8, device=p.device) for p in self.params]
                for _ in range(2))
        self._shapes: Optional[List[torch.Size]] = None

    def _tensors(self, grads: Optional[Sequence[torch.Tensor]] = None) -> int:
        """The descriptors' address; the lists above may have been given other tensors (a checkpoint's), so all are
        looked at."""
        state = torch.float32 if self.bits == 32 else torch.uint8
        params, eight = self.params, self.bits == 8
        shapes = [p.shape for p in params]
        if shapes != self._shapes:
            sizes = [p.numel() for p in params]
            self._shapes, self._scales = shapes, [((n + 127) // 128,) for n in sizes]
            # the library's descriptors, one a row, as the 8 words of ep_adamw_tensor_t
            self._words = np.zeros((len(params), 8), dtype=np.int64)
            self._words[:, 7] = sizes
        words = self._words
        if not all([p.dtype is torch.float32 and p.is_cuda and p.is_contiguous() for p in params]):
            for i, p in enumerate(params):
                _arg_or_raise(p, torch.float32, p.shape, f"params[{i}]")
        if params:
            words[:, 0] = [p.data_ptr() for p in params]
        columns = [(2, self.exp_avg, state, "exp_avg"), (3, self.exp_avg_sq, state, "exp_avg_sq")]
        if grads is not None:
            columns.append((1, grads, grads[0].dtype if grads else torch.float32, "grads"))
            if self.copies is not None:
                columns.append((6, self.copies, torch.bfloat16, "copies"))
            else:
                words[:, 6] = 0
        if eight:
            lengths = self._scales
            columns += [(4, self.exp_avg_scale, torch.uint8, "exp_avg_scale"),
                        (5, self.exp_avg_sq_scale, torch.uint8, "exp_avg_sq_scale")]
        for word, tensors, dtype, name in columns:
            want = lengths if word in (4, 5) else shapes
            if len(tensors) != len(want):
                raise EPBalanceError(f"{name} must be one for each of the {len(want)} parameters")
            if not all([t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous()
                        for t, shape in zip(tensors, want)]):
                for i, (t, shape) in enumerate(zip(tensors, want)):
                    _arg_or_raise(t, dtype, shape, f"{name}[{i}]")
            if want:
                words[:, word] = [t.data_ptr() for t in tensors]
        return words.ctypes.data

    def step(self, grads: Sequence[torch.Tensor], lr: Optional[float] = None, grad_scale: float = 1.0,
             stream=None) -> None:
        """One step; grads fp32 or bf16 (all the same), of the parameters' shapes."""
        dtype = grads[0].dtype if grads else torch.float32
        if dtype not in _FLOATS:
            raise EPBalanceError(f"grads must be float32 or bfloat16, got {dtype}")
        tensors = self._tensors(grads)
        hp = _CAdamW(self.lr if lr is None else lr, self.beta1, self.beta2, self.eps, self.weight_decay, grad_scale,
                     self.step_count + 1, self.seed, self.bits, _FLOATS[dtype])
        rc = lib().ep_adamw_step(tensors, len(self.params), ctypes.byref(hp), _stream(stream))
        _check(rc, "ep_adamw_step")
        self.step_count += 1

    def states(self, stream=None):
        """(exp_avg, exp_avg_sq) as lists of float32 tensors: the moments themselves, or the 8-bit ones' values."""
        if self.bits == 32:
            return self.exp_avg, self.exp_avg_sq
        n = len(self.params)
        if n == 0:
            return [], []
        tensors = self._tensors()
        # the values of all tensors lie one after the other in one piece of memory
        sizes = self._words[:, 7]
        flat = _held(torch.empty((2, int(sizes.sum())), dtype=torch.float32, device=self.params[0].device), stream)
        out = []
        for part in flat.unbind():
            out.append([t if p.dim() == 1 else t.view(p.shape) for t, p in zip(part.split(sizes.tolist()), self.params)])
        mp = flat.data_ptr() + 4 * (np.cumsum(sizes) - sizes)
        vp = mp + 4 * flat.shape[1]
        _check(lib().ep_adamw_values(tensors, n, mp.ctypes.data, vp.ctypes.data, _stream(stream)),
               "ep_adamw_values")
        return out[0], out[1]
