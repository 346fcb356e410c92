"""Binding of the operators around the expert layer: the norms before and after a
block with its gate and residual scales, and expert weights in 4 bits.

Between two blocks of a model, and on into the next one's experts:

    n = block_norm(x, combine(y2, h), weight=w, quantize=True)   # x', h, and h in 8 bits
    g = gate(n.h @ router, K)
    lay = get_dispatch_layout(g.topk_idx, E, P)
    x8, xs, h = dispatch(n.codes, g.topk_weights, lay, use_fp8=True, x_scales=n.scales)
    y1 = grouped_gemm_fp4(x8, xs, w1.codes, w1.scales, h)        # w1 = quantize_weights_fp4(...)
    a8, as_, _, _ = swiglu_fp8(y1, h)
    y2 = grouped_gemm_fp4(a8, as_, w2.codes, w2.scales, h)

Every call enqueues on the current stream of its tensors' device, and returns
without waiting; all its tensors must be on that device.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

from . import _I, _P, _SIGS, _check, _ptr, load
from .experts import _SZ, _group_args, _i32, _matrix, _on, _row_scales, _shape, _stream, _width

EP_GATE_NONE = 0
EP_GATE_TOKEN = 1
EP_GATE_CHANNEL = 2


class ep_block_norm_t(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("y_weight", ctypes.c_void_p),
        ("gate", ctypes.c_void_p),
        ("x_ld", ctypes.c_int64),
        ("y_ld", ctypes.c_int64),
        ("num_rows", ctypes.c_int32),
        ("width", ctypes.c_int32),
        ("x_f32", ctypes.c_int32),
        ("norm", ctypes.c_int32),
        ("y_norm", ctypes.c_int32),
        ("weights_f32", ctypes.c_int32),
        ("gate_kind", ctypes.c_int32),
        ("gate_f32", ctypes.c_int32),
        ("residual_scale", ctypes.c_float),
        ("y_scale", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
    ]


_N = ctypes.POINTER(ep_block_norm_t)
_SIGS.update({
    "ep_block_norm": ([_N, _P, _P, _P, _P, _P], _I),
    "ep_block_norm_workspace_bytes": ([_I, _I], _SZ),
    "ep_block_norm_backward": ([_N, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "ep_quantize_weights_fp4": ([_P, _I, _I, _I, _I, _P, _P, _P], _I),
    "ep_dequantize_weights_fp4": ([_P, _P, _I, _I, _I, _P, _I, _P], _I),
    "ep_grouped_gemm_fp4": ([_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P], _I),
})


# ----------------------------------------------------------------------------
# the C entry points
# ----------------------------------------------------------------------------

def ep_block_norm(args, x_out, h, codes, scales, stream) -> int:
    return load().ep_block_norm(args, x_out, h, codes, scales, stream)


def ep_block_norm_workspace_bytes(num_rows: int, width: int) -> int:
    return load().ep_block_norm_workspace_bytes(num_rows, width)


def ep_block_norm_backward(args, grad_x, grad_h, out_x, out_y, out_weight, out_y_weight, out_gate, ws,
                           ws_bytes, stream) -> int:
    return load().ep_block_norm_backward(args, grad_x, grad_h, out_x, out_y, out_weight, out_y_weight,
                                         out_gate, ws, ws_bytes, stream)


def ep_quantize_weights_fp4(w, w_f32, num_groups, n, k, codes, scales, stream) -> int:
    return load().ep_quantize_weights_fp4(w, int(w_f32), num_groups, n, k, codes, scales, stream)


def ep_dequantize_weights_fp4(codes, scales, num_groups, n, k, out, out_f32, stream) -> int:
    return load().ep_dequantize_weights_fp4(codes, scales, num_groups, n, k, out, int(out_f32), stream)


def ep_grouped_gemm_fp4(x, x_scales, scale_ld, w, w_scales, group_offsets, num_groups, group_stride,
                        num_rows, n, k, expected_rows, out, stream) -> int:
    return load().ep_grouped_gemm_fp4(x, x_scales, scale_ld, w, w_scales, group_offsets, num_groups,
                                      group_stride, num_rows, n, k, expected_rows, out, stream)


# ----------------------------------------------------------------------------
# the same calls on torch tensors
# ----------------------------------------------------------------------------

def _rows(t, T, H, name):
    """Elements between the rows of a matrix [T, H] whose rows are contiguous (they may lie apart)."""
    ld, step = (H, 1) if t.is_contiguous() else t.stride()
    if T <= 1:
        ld = H
    if step != 1 and T > 0 and H > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if ld < H or ld % 8:
        raise ValueError(f"{name}: the stride of its rows ({ld}) must be a multiple of 8 and at least {H}")
    return ld


def _f32(t, name):
    """Whether a tensor that may be bf16 or fp32 is fp32."""
    import torch
    if t.dtype is torch.float32:
        return 1
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return 0


def _norm_args(x, y, norm, weight, y_norm, y_weight, gate, residual_scale, y_scale, eps, weight_offset):
    import torch
    T, H = shape = _matrix(x, "x")
    if H >= 2 ** 31:
        _i32(H, "width")
    yp = wp = ywp = gp = None
    y_ld = weights_f32 = kind = gate_f32 = 0
    x_f32 = _f32(x, "x")
    x_ld = _rows(x, T, H, "x")
    if y is not None:
        if y.shape != shape:
            _shape(y, (T, H), "y")
        if y.dtype is not torch.bfloat16:
            raise TypeError(f"y must be torch.bfloat16, got {y.dtype}")
        yp, y_ld = y.data_ptr(), _rows(y, T, H, "y")
    elif y_norm or y_weight is not None or gate is not None or residual_scale != 1.0 or not norm:
        raise ValueError("without y there is a norm of x alone: y_norm, y_weight, gate and residual_scale need y")
    if weight is not None:
        if not norm:
            raise ValueError("weight needs norm")
        _shape(weight, (H,), "weight")
        weights_f32 = _f32(weight, "weight")
        wp = _ptr(weight, None, "weight")
    if y_weight is not None:
        _shape(y_weight, (H,), "y_weight")
        weights_f32 = _f32(y_weight, "y_weight")
        if weight is not None and weight.dtype is not y_weight.dtype:
            raise TypeError(f"weight and y_weight must be of one type, got {weight.dtype} and {y_weight.dtype}")
        ywp = _ptr(y_weight, None, "y_weight")
    if gate is not None:
        kind = EP_GATE_TOKEN if gate.shape == (T, 1) else EP_GATE_CHANNEL
        if kind == EP_GATE_CHANNEL and gate.shape != (1, H):
            raise ValueError(f"gate must be [{T}, 1] or [1, {H}], got shape {list(gate.shape)}")
        gate_f32 = _f32(gate, "gate")
        gp = _ptr(gate, None, "gate")
    return ep_block_norm_t(x.data_ptr(), yp, wp, ywp, gp, x_ld, y_ld, T, H, x_f32, bool(norm), bool(y_norm),
                           weights_f32, kind, gate_f32, residual_scale, y_scale, eps, weight_offset), T, H


def _empty(t, dtype=None):
    """A dense tensor of t's shape (empty_like costs the host two thirds of what empty does)."""
    import torch
    if dtype is None and t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _written(t):
    """Tells autograd that a call wrote into a tensor of the caller's, as torch's own in-place
    operations do: a backward pass that kept it raises instead of reading the new values."""
    import torch
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


def _at(t):
    """Address of a tensor that the call itself made."""
    return None if t is None else t.data_ptr()


@dataclass
class BlockNorm:
    """What a block norm gives: the new residual stream (x itself without y), its
    norm in bf16, and the norm as FP8 rows, which ``dispatch`` takes as x, x_scales."""
    x: object
    h: object = None
    codes: object = None
    scales: object = None


def block_norm(x, y=None, *, norm: bool = True, weight=None, y_norm: bool = False, y_weight=None, gate=None,
               residual_scale: float = 1.0, y_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0,
               quantize: bool = False, write_h: bool = True, x_out=None) -> BlockNorm:
    """The norms before and after a block, in one pass over the rows.

    x: the residual stream, bf16 or fp32 [T, H]; y: a block's output (combine's),
    bf16 [T, H], or None.  Rows may lie apart (a stride that is a multiple of 8);
    H is a multiple of 8 (of 128 with quantize).

        z  = y / sqrt(mean(y^2) + eps)  (with y_norm; else y)
        x' = residual_scale * x + y_scale * gate * z * (weight_offset + y_weight)
        h  = x' / sqrt(mean(x'^2) + eps) * (weight_offset + weight)

    weight, y_weight: bf16 or fp32 [H], or None (no factor); gate: bf16 or fp32, one
    factor a token [T, 1] or a channel [1, H], or None.  Returns ``BlockNorm``: x'
    of x's type, h in bf16 (with norm and write_h), and with quantize the same as
    FP8 rows.  x_out may be given, x itself for an update in place."""
    import torch
    with _on(x, y, weight, y_weight, gate, x_out):
        a, T, H = _norm_args(x, y, norm, weight, y_norm, y_weight, gate, residual_scale, y_scale, eps,
                             weight_offset)
        if quantize and not norm:
            raise ValueError("quantize needs norm")
        given = False
        if x_out is not None:
            if y is None:
                raise ValueError("x_out needs y: without it x' is x")
            _shape(x_out, (T, H), "x_out")
            if x_out.dtype is not x.dtype:
                raise TypeError(f"x_out must be {x.dtype}, got {x_out.dtype}")
            given = True
        elif y is not None:
            x_out = _empty(x)
        h = codes = scales = None
        if norm and write_h:
            h = _empty(x, None if x.dtype is torch.bfloat16 else torch.bfloat16)
        if quantize:
            codes = _empty(x, torch.float8_e4m3fn)
            scales = torch.empty_strided((T, H // 128), (H // 128, 1), dtype=torch.float32, device=x.device)
        _check(ep_block_norm(a, _ptr(x_out, None, "x_out"), _at(h), _at(codes) if T else None,
                             _at(scales) if T else None, _stream(x)))
        if given:
            _written(x_out)
    return BlockNorm(x if y is None else x_out, h, codes, scales)


@dataclass
class BlockNormGrads:
    """Gradients of a block norm's inputs (None: not asked for, or no such input)."""
    x: object = None
    y: object = None
    weight: object = None
    y_weight: object = None
    gate: object = None


_INPUTS = ("x", "y", "weight", "y_weight", "gate")


def block_norm_backward(x, y=None, *, grad_x=None, grad_h=None, norm: bool = True, weight=None,
                        y_norm: bool = False, y_weight=None, gate=None, residual_scale: float = 1.0,
                        y_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0,
                        need=_INPUTS, ws=None) -> BlockNormGrads:
    """Gradients of ``block_norm``'s inputs, from the same inputs and options.

    grad_x: gradient of x' (the residual stream's, x's type) or None; grad_h: gradient
    of h (bf16) or None; both [T, H] and contiguous.  need: which gradients to write.
    Each has its input's shape and type.  ws (uint8, >= ep_block_norm_workspace_bytes(T,
    H)) may be passed to reuse a workspace."""
    import torch
    bad = [n for n in need if n not in _INPUTS]
    if bad:
        raise ValueError(f"need holds {bad[0]!r}: it may hold {list(_INPUTS)}")
    with _on(x, y, weight, y_weight, gate, grad_x, grad_h, ws):
        a, T, H = _norm_args(x, y, norm, weight, y_norm, y_weight, gate, residual_scale, y_scale, eps,
                             weight_offset)
        if grad_x is not None:
            _shape(grad_x, (T, H), "grad_x")
            if grad_x.dtype != x.dtype:
                raise TypeError(f"grad_x must be {x.dtype}, got {grad_x.dtype}")
        if grad_h is not None:
            if not norm:
                raise ValueError("grad_h needs norm")
            _shape(grad_h, (T, H), "grad_h")

        def new(t, name):
            if t is None or name not in need:
                return None
            return _empty(t)

        o = BlockNormGrads(new(x, "x"), new(y, "y"), new(weight, "weight"), new(y_weight, "y_weight"),
                           new(gate, "gate"))
        columns = o.weight is not None or o.y_weight is not None
        columns = columns or (o.gate is not None and a.gate_kind == EP_GATE_CHANNEL)
        if not columns:
            ws = None
        elif ws is None:
            ws = torch.empty(ep_block_norm_workspace_bytes(T, H), dtype=torch.uint8, device=x.device)
        if columns or (T > 0 and (o.x is not None or o.y is not None or o.gate is not None)):
            _check(ep_block_norm_backward(a, _ptr(grad_x, None, "grad_x"), _ptr(grad_h, "bf16", "grad_h"),
                                          _at(o.x), _at(o.y), _at(o.weight), _at(o.y_weight), _at(o.gate),
                                          _ptr(ws, "u8", "ws"), 0 if ws is None else ws.numel(), _stream(x)))
    return o


@dataclass
class Fp4Weights:
    """Expert weights in 4 bits: codes (two in a byte) uint8 [G, N, K/2] and scales
    float8_e8m0fnu [G, N, K/32]."""
    codes: object
    scales: object


def quantize_weights_fp4(w) -> Fp4Weights:
    """w: bf16 or fp32 [G, N, K], N and K multiples of 128.  E2M1 codes, an even k in
    a byte's low half, with one power of two for 32 weights along K."""
    import torch
    if w.dim() != 3:
        raise ValueError(f"w must be [G, N, K], got shape {list(w.shape)}")
    f32 = _f32(w, "w")
    G, N, K = w.shape
    _width(N, "N")
    _width(K, "K")
    with _on(w):
        codes = torch.empty((G, N, K // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((G, N, K // 32), dtype=torch.float8_e8m0fnu, device=w.device)
        _check(ep_quantize_weights_fp4(_ptr(w, name="w"), f32, _i32(G, "G"), N, K, _at(codes), _at(scales),
                                       _stream(w)))
    return Fp4Weights(codes, scales)


def _fp4_shape(w, w_scales):
    if w.dim() != 3:
        raise ValueError(f"w must be [G, N, K/2], got shape {list(w.shape)}")
    G, N, K = w.shape
    K *= 2
    if N % 128 or K % 128 or not (0 < N < 2 ** 31 and 0 < K < 2 ** 31):
        _width(N, "N")
        _width(K, "K")
    _shape(w_scales, (G, N, K // 32), "w_scales")
    return G, N, K


def dequantize_weights_fp4(w: Fp4Weights, dtype=None):
    """The values that 4-bit weights stand for, [G, N, K] in torch.bfloat16 (default) or
    torch.float32, exactly."""
    import torch
    G, N, K = _fp4_shape(w.codes, w.scales)
    with _on(w.codes, w.scales):
        out = torch.empty((G, N, K), dtype=dtype or torch.bfloat16, device=w.codes.device)
        f32 = _f32(out, "dtype")
        _check(ep_dequantize_weights_fp4(_ptr(w.codes, "fp4", "codes"), _ptr(w.scales, "e8m0", "scales"),
                                         _i32(G, "G"), N, K, _at(out), f32, _stream(out)))
    return out


def grouped_gemm_fp4(x, x_scales, w, w_scales, groups, *, group_stride: int = 0, expected_rows: int = 0,
                     column_major_scales: bool = False, out=None):
    """The experts' product on FP8 rows with 4-bit weights: ``grouped_gemm_fp8`` with w,
    w_scales from ``quantize_weights_fp4`` (codes [G, N, K/2], scales [G, N, K/32]).
    out[r] = x[r] @ w[g].T for the rows r of group g, bf16 [rows, N]."""
    import torch
    rows, K = _matrix(x, "x")
    G, N, k = _fp4_shape(w, w_scales)
    if k != K:
        raise ValueError(f"w must be [G, N, {K // 2}], got shape {list(w.shape)}")
    ld = _row_scales(x_scales, rows, K, column_major_scales, "x_scales")
    if group_stride or expected_rows:
        group_stride, expected_rows = _i32(group_stride, "group_stride"), _i32(expected_rows, "expected_rows")
    with _on(x, x_scales, w, w_scales, out):
        args, expected = _group_args(groups, group_stride, x)
        if args[1] != G:
            raise ValueError(f"w holds {G} groups, the rows {args[1]}")
        given = out is not None
        if not given:
            out = torch.empty((rows, N), dtype=torch.bfloat16, device=x.device)
        elif out.shape != (rows, N):
            _shape(out, (rows, N), "out")
        _check(ep_grouped_gemm_fp4(_ptr(x, "fp8", "x"), _ptr(x_scales, "f32", "x_scales"), ld,
                                   _ptr(w, "fp4", "w"), _ptr(w_scales, "e8m0", "w_scales"), *args, rows, N, K,
                                   expected_rows or expected, _ptr(out, "bf16", "out"), _stream(x)))
        if given:
            _written(out)
    return out
