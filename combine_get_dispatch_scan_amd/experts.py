"""Binding of the expert layer: the gate, the FP8 quantisers, the grouped FP8
product, its weight gradient, and SwiGLU with an 8-bit checkpoint.

One layer, as these calls and dispatch / combine make it up:

    g = gate(logits, K, balance_coef=1e-2)                    # ids, weights, loss
    lay = get_dispatch_layout(g.topk_idx, E, P)
    x8, xs, h = dispatch(x, g.topk_weights, lay, use_fp8=True)
    y1 = grouped_gemm_fp8(x8, xs, w1.codes, w1.scales, h)     # [rows, 2 * inner]
    a8, as_, c8, cs = swiglu_fp8(y1, h, checkpoint=True)
    y2 = grouped_gemm_fp8(a8, as_, w2.codes, w2.scales, h)
    out = combine(y2, h)

``groups`` says which rows belong to which expert: a dispatched ``Handle`` (any
layout), or an int32 GPU tensor [G + 1] of row offsets (with ``group_stride`` for
a static layout: group g's rows begin at g * group_stride).  Rows of no group are
neither read nor written: in outputs that the call allocates they are undefined.

Every call enqueues on the current stream of its tensors' device, and returns
without waiting; all its tensors must be on that device.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional

from . import _I, _P, _SIGS, Handle, _check, _ptr, load

EP_GATE_SOFTMAX = 0
EP_GATE_SIGMOID = 1

_SZ = ctypes.c_size_t
_F = ctypes.c_float
_L = ctypes.c_int64
_SIGS.update({
    "ep_gate_workspace_bytes": ([_I, _I], _SZ),
    "ep_gate": ([_P, _I, _L, _I, _I, _I, _I, _I, _F, _F, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "ep_gate_backward": ([_P, _I, _L, _I, _I, _I, _I, _I, _F, _F, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "ep_quantize_rows": ([_P, _I, _P, _I, _I, _I, _I, _P, _P, _P], _I),
    "ep_quantize_weights": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "ep_grouped_gemm_fp8": ([_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P], _I),
    "ep_grouped_wgrad_fp8": ([_P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _P, _I, _P], _I),
    "ep_swiglu_fp8": ([_P, _I, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "ep_swiglu_fp8_backward": ([_P, _P, _P, _I, _P, _I, _I, _I, _I, _P, _P, _P, _P], _I),
})


# ----------------------------------------------------------------------------
# the C entry points
# ----------------------------------------------------------------------------

def ep_gate_workspace_bytes(num_tokens: int, num_experts: int) -> int:
    return load().ep_gate_workspace_bytes(num_tokens, num_experts)


def ep_gate(logits, logits_bf16, ld, num_tokens, num_experts, num_topk, score, normalize, scale,
            balance_coef, token_mask, topk_idx, topk_weights, num_tokens_per_expert, num_valid, loss,
            ws, ws_bytes, stream) -> int:
    return load().ep_gate(logits, int(logits_bf16), ld, num_tokens, num_experts, num_topk, score,
                          int(normalize), scale, balance_coef, token_mask, topk_idx, topk_weights,
                          num_tokens_per_expert, num_valid, loss, ws, ws_bytes, stream)


def ep_gate_backward(logits, logits_bf16, ld, num_tokens, num_experts, num_topk, score, normalize, scale,
                     balance_coef, token_mask, topk_idx, num_tokens_per_expert, num_valid, grad_weights,
                     grad_loss, grad_logits, stream) -> int:
    return load().ep_gate_backward(logits, int(logits_bf16), ld, num_tokens, num_experts, num_topk, score,
                                   int(normalize), scale, balance_coef, token_mask, topk_idx,
                                   num_tokens_per_expert, num_valid, grad_weights, grad_loss, grad_logits,
                                   stream)


def ep_quantize_rows(x, width, group_offsets, num_groups, group_stride, num_rows, scale_ld, codes, scales,
                     stream) -> int:
    return load().ep_quantize_rows(x, width, group_offsets, num_groups, group_stride, num_rows, scale_ld,
                                   codes, scales, stream)


def ep_quantize_weights(w, w_f32, num_groups, n, k, codes, scales, codes_t, scales_t, stream) -> int:
    return load().ep_quantize_weights(w, int(w_f32), num_groups, n, k, codes, scales, codes_t, scales_t,
                                      stream)


def ep_grouped_gemm_fp8(x, x_scales, scale_ld, w, w_scales, group_offsets, num_groups, group_stride,
                        num_rows, n, k, expected_rows, out, stream) -> int:
    return load().ep_grouped_gemm_fp8(x, x_scales, scale_ld, w, w_scales, group_offsets, num_groups,
                                      group_stride, num_rows, n, k, expected_rows, out, stream)


def ep_grouped_wgrad_fp8(grad, x, x_scales, scale_ld, group_offsets, num_groups, group_stride, num_rows, n,
                         k, out, out_f32, stream) -> int:
    return load().ep_grouped_wgrad_fp8(grad, x, x_scales, scale_ld, group_offsets, num_groups, group_stride,
                                       num_rows, n, k, out, int(out_f32), stream)


def ep_swiglu_fp8(h, inner, group_offsets, num_groups, group_stride, num_rows, scale_ld, codes, scales,
                  ckpt, ckpt_scales, stream) -> int:
    return load().ep_swiglu_fp8(h, inner, group_offsets, num_groups, group_stride, num_rows, scale_ld,
                                codes, scales, ckpt, ckpt_scales, stream)


def ep_swiglu_fp8_backward(grad_a, ckpt, ckpt_scales, inner, group_offsets, num_groups, group_stride,
                           num_rows, scale_ld, grad_h, codes, scales, stream) -> int:
    return load().ep_swiglu_fp8_backward(grad_a, ckpt, ckpt_scales, inner, group_offsets, num_groups,
                                         group_stride, num_rows, scale_ld, grad_h, codes, scales, stream)


# ----------------------------------------------------------------------------
# the same calls on torch tensors
# ----------------------------------------------------------------------------

@contextlib.contextmanager
def _device_of(dev):
    import torch
    with torch.cuda.device(dev):
        yield


_HERE = contextlib.nullcontext()


def _on(t, *others):
    """A context in which t's device is current; every other tensor must be on it."""
    import torch
    if not t.is_cuda:
        raise ValueError(f"expected GPU tensors (got device {t.device})")
    for o in others:
        if o is not None and o.device != t.device:
            raise ValueError(f"all tensors must be on one device (got {t.device} and {o.device})")
    return _HERE if t.device.index == torch.cuda.current_device() else _device_of(t.device)


def _stream(t):
    import torch
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _shape(t, want, name):
    if t.shape != want:
        raise ValueError(f"{name} must have shape {list(want)}, got {list(t.shape)}")


def _i32(n, name):
    """n as the int the C call takes it as (ctypes would cut higher bits off)."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name}={n} must be less than 2^31")
    return int(n)


def _width(n, name):
    if _i32(n, name) < 128 or n % 128:
        raise ValueError(f"{name}={n} must be a multiple of 128")


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix [rows, width], got shape {list(t.shape)}")
    _i32(t.shape[0], "rows")
    return t.shape


def _groups(groups, group_stride, like):
    """(offsets tensor, number of groups, stride, expected rows of a group or 0)"""
    if isinstance(groups, Handle):
        c = groups.c
        if group_stride:
            raise ValueError("group_stride is taken from the handle")
        off = groups.expert_offset
        expected = -(-c.num_tokens * c.num_topk // c.num_experts)
        return off, c.num_experts, c.static_cap, max(1, expected)
    if groups.dim() != 1 or groups.numel() < 2:
        raise ValueError(f"groups must be a Handle or row offsets [num_groups + 1], got shape {list(groups.shape)}")
    return groups, _i32(groups.numel() - 1, "num_groups"), group_stride, 0


def _group_args(groups, group_stride, like):
    off, n, stride, expected = _groups(groups, group_stride, like)
    if off.device != like.device:
        raise ValueError(f"all tensors must be on one device (got {like.device} and {off.device})")
    return (_ptr(off, "i32", "groups"), n, stride), expected


def _row_scales(scales, rows, width, column_major, name):
    """Leading dimension of row scales (0: row-major), their shape checked."""
    if column_major:
        if scales.dim() != 2 or scales.shape[0] != width // 128 or scales.shape[1] < rows or scales.shape[1] % 4:
            raise ValueError(f"{name} must have shape [{width // 128}, ld] with ld >= {rows} and a multiple "
                             f"of 4 (column-major), got {list(scales.shape)}")
        return scales.shape[1]
    _shape(scales, (rows, width // 128), name)
    return 0


def _new_rows(rows, width, column_major, dev):
    """Codes and scales of FP8 rows that a call writes, and the scales' leading dimension."""
    import torch
    codes = torch.empty((rows, width), dtype=torch.float8_e4m3fn, device=dev)
    ld = max(4, (rows + 3) // 4 * 4) if column_major else 0
    shape = (width // 128, ld) if column_major else (rows, width // 128)
    return codes, torch.empty(shape, dtype=torch.float32, device=dev), ld


@dataclass
class Gate:
    """What the gate chose, and what its backward pass needs besides the logits."""
    topk_idx: object                # int64 [T, K], -1 where no expert was left
    topk_weights: object            # fp32 [T, K]
    num_tokens_per_expert: object   # int32 [E]
    num_valid: object               # int32 [1], tokens that count
    loss: object                    # fp32 [1], the balance loss
    score: int
    normalize: bool
    scale: float
    balance_coef: float
    token_mask: object


_SCORES = {"softmax": EP_GATE_SOFTMAX, "sigmoid": EP_GATE_SIGMOID}


def _logits(logits):
    """(T, E, whether bf16, elements between rows)"""
    import torch
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, E], got shape {list(logits.shape)}")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be torch.float32 or torch.bfloat16, got {logits.dtype}")
    T, E = logits.shape
    _i32(T, "tokens")
    _i32(E, "experts")
    if T > 0 and E > 1 and logits.stride(1) != 1:
        raise ValueError("the logits of a token must be contiguous")
    ld = logits.stride(0) if T > 1 else E
    if ld < E:
        raise ValueError(f"rows of logits must not overlap (stride {ld} < {E})")
    return T, E, logits.dtype == torch.bfloat16, ld


def gate(logits, num_topk: int, *, score: str = "softmax", normalize: bool = True, scale: float = 1.0,
         balance_coef: float = 0.0, token_mask=None, ws=None) -> Gate:
    """logits: fp32 or bf16 [T, E] on the GPU (rows may be strided).  Chooses each
    token's num_topk largest logits (ties to the lower id; a logit of -inf is
    never chosen) and returns ids, weights, the pairs per expert and the balance
    loss (``Gate``).  score "softmax" or "sigmoid"; normalize divides a token's
    weights by their sum, scale multiplies them.  token_mask (uint8 or bool [T]):
    tokens with 0 get ids -1 and count nowhere.  ws (uint8, >=
    ep_gate_workspace_bytes(T, E)) may be passed to reuse a workspace."""
    import torch
    T, E, bf16, ld = _logits(logits)
    K = max(_i32(num_topk, "num_topk"), 0)
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if token_mask is not None:
        _shape(token_mask, (T,), "token_mask")
        if token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
    dev = logits.device
    with _on(logits, token_mask, ws):
        idx = torch.empty((T, K), dtype=torch.int64, device=dev)
        w = torch.empty((T, K), dtype=torch.float32, device=dev)
        # storage of their own: a kept loss holds no workspace, and torch counts changes of each by itself
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        valid = torch.empty(1, dtype=torch.int32, device=dev)
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        if ws is None:
            ws = torch.empty(ep_gate_workspace_bytes(T, E), dtype=torch.uint8, device=dev)
        _check(ep_gate(logits.data_ptr(), bf16, ld, T, E, K, _SCORES[score], bool(normalize), scale,
                       balance_coef, _ptr(token_mask, "u8", "token_mask"), idx.data_ptr(), w.data_ptr(),
                       counts.data_ptr(), valid.data_ptr(), loss.data_ptr(), _ptr(ws, "u8", "ws"), ws.numel(),
                       _stream(logits)))
    return Gate(idx, w, counts, valid, loss, _SCORES[score], bool(normalize), float(scale),
                float(balance_coef), token_mask)


def gate_backward(logits, g: Gate, grad_weights=None, grad_loss=None):
    """Gradient of sum(grad_weights * topk_weights) + grad_loss * loss towards the
    logits (the ones the gate was given): [T, E], dense, of their type.
    grad_weights: fp32 [T, K] or None; grad_loss: fp32 with one value, or None."""
    import torch
    T, E, bf16, ld = _logits(logits)
    K = g.topk_idx.shape[1]
    _shape(g.topk_idx, (T, K), "topk_idx")
    _shape(g.num_tokens_per_expert, (E,), "num_tokens_per_expert")
    _shape(g.num_valid, (1,), "num_valid")
    if g.token_mask is not None:
        _shape(g.token_mask, (T,), "token_mask")
    if grad_weights is not None:
        _shape(grad_weights, (T, K), "grad_weights")
    if grad_loss is not None and grad_loss.numel() != 1:
        raise ValueError(f"grad_loss must hold one value, got shape {list(grad_loss.shape)}")
    with _on(logits, g.topk_idx, g.num_tokens_per_expert, g.num_valid, g.token_mask, grad_weights, grad_loss):
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
        _check(ep_gate_backward(logits.data_ptr(), bf16, ld, T, E, K, g.score, g.normalize, g.scale,
                                g.balance_coef, _ptr(g.token_mask, "u8", "token_mask"),
                                _ptr(g.topk_idx, "i64", "topk_idx"),
                                _ptr(g.num_tokens_per_expert, "i32", "num_tokens_per_expert"),
                                _ptr(g.num_valid, "i32", "num_valid"),
                                _ptr(grad_weights, "f32", "grad_weights"),
                                _ptr(grad_loss, "f32", "grad_loss"), _ptr(out), _stream(logits)))
    return out


def quantize_rows(x, groups=None, *, group_stride: int = 0, column_major_scales: bool = False):
    """x: bf16 [rows, H], H % 128 == 0.  Returns FP8 rows (codes float8_e4m3fn
    [rows, H], scales fp32 [rows, H/128], or [H/128, ld] column-major).  groups
    None: every row; else only rows of a group."""
    rows, H = _matrix(x, "x")
    _width(H, "H")
    group_stride = _i32(group_stride, "group_stride")
    with _on(x):
        args, _ = ((None, 0, 0), 0) if groups is None else _group_args(groups, group_stride, x)
        codes, scales, ld = _new_rows(rows, H, column_major_scales, x.device)
        _check(ep_quantize_rows(_ptr(x, "bf16", "x"), H, *args, rows, ld, _ptr(codes), _ptr(scales),
                                _stream(x)))
    return codes, scales


@dataclass
class Fp8Weights:
    """Expert weights in 8 bits: codes [G, N, K], scales [G, N/128, K/128], and,
    when asked for, the transposed ones [G, K, N] that the product towards the
    input reads."""
    codes: object
    scales: object
    codes_t: object = None
    scales_t: object = None


def quantize_weights(w, transposed: bool = False) -> Fp8Weights:
    """w: bf16 or fp32 [G, N, K], N and K multiples of 128.  One scale per 128 x 128
    block; transposed also writes the transposed codes and scales."""
    import torch
    if w.dim() != 3:
        raise ValueError(f"w must be [G, N, K], got shape {list(w.shape)}")
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"w must be torch.bfloat16 or torch.float32, got {w.dtype}")
    G, N, K = w.shape
    _width(N, "N")
    _width(K, "K")
    with _on(w):
        new = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=w.device)  # noqa: E731
        f8 = torch.float8_e4m3fn
        o = Fp8Weights(new(G, N, K, dt=f8), new(G, N // 128, K // 128))
        if transposed:
            o.codes_t, o.scales_t = new(G, K, N, dt=f8), new(G, K // 128, N // 128)
        _check(ep_quantize_weights(_ptr(w, name="w"), w.dtype == torch.float32, G, N, K, _ptr(o.codes),
                                   _ptr(o.scales), _ptr(o.codes_t), _ptr(o.scales_t), _stream(w)))
    return o


def grouped_gemm_fp8(x, x_scales, w, w_scales, groups, *, group_stride: int = 0, expected_rows: int = 0,
                     column_major_scales: bool = False, out=None):
    """The experts' product on FP8 rows: out[r] = x[r] @ w[g].T for the rows r of
    group g, bf16 [rows, N].  x: codes [rows, K] with their scales as dispatch or
    the quantisers wrote them; w, w_scales: an expert-major ``Fp8Weights`` pair
    (codes, scales, or codes_t, scales_t for the gradient towards the input).
    expected_rows: typical rows of a group (a handle knows it; otherwise rows /
    groups); it chooses the tile.  out may be given; rows of no group keep what
    they held."""
    import torch
    rows, K = _matrix(x, "x")
    if w.dim() != 3 or w.shape[2] != K:
        raise ValueError(f"w must be [G, N, {K}], got shape {list(w.shape)}")
    G, N = w.shape[0], w.shape[1]
    _width(K, "K")
    _width(N, "N")
    _shape(w_scales, (G, N // 128, K // 128), "w_scales")
    ld = _row_scales(x_scales, rows, K, column_major_scales, "x_scales")
    group_stride, expected_rows = _i32(group_stride, "group_stride"), _i32(expected_rows, "expected_rows")
    with _on(x, x_scales, w, w_scales, out):
        args, expected = _group_args(groups, group_stride, x)
        if args[1] != G:
            raise ValueError(f"w holds {G} groups, the rows {args[1]}")
        if out is None:
            out = torch.empty((rows, N), dtype=torch.bfloat16, device=x.device)
        _shape(out, (rows, N), "out")
        _check(ep_grouped_gemm_fp8(_ptr(x, "fp8", "x"), _ptr(x_scales, "f32", "x_scales"), ld,
                                   _ptr(w, "fp8", "w"), _ptr(w_scales, "f32", "w_scales"), *args, rows, N, K,
                                   expected_rows or expected, _ptr(out, "bf16", "out"), _stream(x)))
    return out


def grouped_wgrad_fp8(grad, x, x_scales, groups, *, group_stride: int = 0, out_dtype=None,
                      column_major_scales: bool = False, out=None):
    """Weight gradient of the product: out[g] = grad[rows of g].T @ x[rows of g],
    [G, N, K], from grad bf16 [rows, N] and the product's FP8 input rows.
    out_dtype torch.bfloat16 (default) or torch.float32; groups without rows get 0."""
    import torch
    rows, K = _matrix(x, "x")
    N = _matrix(grad, "grad")[1]
    _shape(grad, (rows, N), "grad")
    _width(K, "K")
    _width(N, "N")
    ld = _row_scales(x_scales, rows, K, column_major_scales, "x_scales")
    group_stride = _i32(group_stride, "group_stride")
    with _on(x, grad, x_scales, out):
        args, _ = _group_args(groups, group_stride, x)
        if out is None:
            out = torch.empty((args[1], N, K), dtype=out_dtype or torch.bfloat16, device=x.device)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
        _shape(out, (args[1], N, K), "out")
        if out.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"out must be torch.bfloat16 or torch.float32, got {out.dtype}")
        _check(ep_grouped_wgrad_fp8(_ptr(grad, "bf16", "grad"), _ptr(x, "fp8", "x"),
                                    _ptr(x_scales, "f32", "x_scales"), ld, *args, rows, N, K,
                                    _ptr(out, name="out"), out.dtype == torch.float32, _stream(x)))
    return out


def swiglu_fp8(h, groups=None, *, group_stride: int = 0, checkpoint: bool = False,
               column_major_scales: bool = False):
    """h = [g | u], bf16 [rows, 2 * inner].  Returns (codes, scales, ckpt,
    ckpt_scales): silu(g) * u as FP8 rows of width inner, and, with checkpoint, h
    itself as FP8 rows for ``swiglu_fp8_backward`` (else None, None)."""
    rows, W = _matrix(h, "h")
    inner = W // 2
    if W % 2:
        raise ValueError(f"h must be [rows, 2 * inner], got shape {list(h.shape)}")
    _width(inner, "inner")
    group_stride = _i32(group_stride, "group_stride")
    with _on(h):
        args, _ = ((None, 0, 0), 0) if groups is None else _group_args(groups, group_stride, h)
        codes, scales, ld = _new_rows(rows, inner, column_major_scales, h.device)
        ck = cs = None
        if checkpoint:
            ck, cs, _ = _new_rows(rows, W, False, h.device)
        # a call without rows has nothing to write (torch gives empty tensors no address)
        _check(ep_swiglu_fp8(_ptr(h, "bf16", "h"), inner, *args, rows, ld, _ptr(codes), _ptr(scales),
                             _ptr(ck) if rows else None, _ptr(cs) if rows else None, _stream(h)))
    return codes, scales, ck, cs


def swiglu_fp8_backward(grad_a, ckpt, ckpt_scales, groups=None, *, group_stride: int = 0,
                        quantize: bool = True, column_major_scales: bool = False):
    """Gradient of SwiGLU towards h from its 8-bit checkpoint.  grad_a: bf16 [rows,
    inner].  Returns (grad_h bf16 [rows, 2 * inner], and the same as FP8 rows:
    codes, scales; None, None without quantize)."""
    import torch
    rows, inner = _matrix(grad_a, "grad_a")
    _width(inner, "inner")
    _shape(ckpt, (rows, 2 * inner), "ckpt")
    _shape(ckpt_scales, (rows, 2 * inner // 128), "ckpt_scales")
    group_stride = _i32(group_stride, "group_stride")
    with _on(grad_a, ckpt, ckpt_scales):
        args, _ = ((None, 0, 0), 0) if groups is None else _group_args(groups, group_stride, grad_a)
        grad_h = torch.empty((rows, 2 * inner), dtype=torch.bfloat16, device=grad_a.device)
        codes = scales = None
        ld = 0
        if quantize:
            codes, scales, ld = _new_rows(rows, 2 * inner, column_major_scales, grad_a.device)
        _check(ep_swiglu_fp8_backward(_ptr(grad_a, "bf16", "grad_a"), _ptr(ckpt, "fp8", "ckpt"),
                                      _ptr(ckpt_scales, "f32", "ckpt_scales"), inner, *args, rows, ld,
                                      _ptr(grad_h), _ptr(codes) if rows else None,
                                      _ptr(scales) if rows else None, _stream(grad_a)))
    return grad_h, codes, scales
