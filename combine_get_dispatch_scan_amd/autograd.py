"""Autograd wrappers of dispatch and combine for training.

The backward of dispatch is combine and the backward of combine is dispatch
(stakiran github-trend-summarizer, "DeepEP 要約", section 3), so each
Function's backward is one of the library's backward calls on the forward's
handle:

    recv, handle = dispatch(x, topk_idx, topk_weights, E, P)   # BF16 rows
    out = combine(y, handle, topk_weights)                     # y: expert outputs

dispatch's backward is ep_dispatch_backward (the unit-weight combine of the
received rows' gradients); combine's backward is ep_combine_backward
(weight-scaled rows of grad_out, and the weight gradient when topk_weights
requires grad).  Receive rows that no pair maps to get a zero gradient.
``gate`` and ``experts`` do the same for the rest of an MoE layer:

    g = gate(logits, K, balance_coef=1e-2)          # ids; weights and loss with gradients
    out = experts(x, g.topk_idx, g.topk_weights, w1, w2, P)
    (task_loss(out) + g.loss).backward()

and ``block_norm`` for what lies between two layers, with gradients of the residual
stream, the block's output, the norms' weights and the gate:

    n = block_norm(x, out, weight=w)                           # n.x: the new stream, n.h: its norm

``experts`` is dispatch, the two FP8 products with SwiGLU between them, and
combine.  It keeps what the wanted gradients read: activations in 8 bits (the
dispatched rows, SwiGLU's input and output), and, only where topk_weights needs
a gradient, the second product's output in bf16.  Its gradient rows are
quantised the same way for the products towards the inputs; the quantisers are
taken as straight-through.  The weights are quantised in every call: inference
with constant weights keeps ``quantize_weights``'s result and makes the plain
calls.

Only argument marshalling happens here; every step runs in the HIP kernels.
These functions are for eager autograd: a backward pass captured into a graph
while an eager graph of the same leaves is alive ends the process in torch, so
``gate``, ``experts`` and ``block_norm`` refuse to be captured, forward and backward (the plain
calls they are made of can be).  None of them has a second derivative: asking for one raises.
"""
from __future__ import annotations

import dataclasses
import functools

import torch

from . import combine as _combine
from . import combine_backward as _combine_backward
from . import dispatch as _dispatch
from . import dispatch_backward as _dispatch_backward
from . import gate as _gate_call
from . import gate_backward as _gate_backward
from . import get_dispatch_layout as _get_dispatch_layout
from . import block_norm as _block_norm_call
from . import block_norm_backward as _block_norm_backward
from . import (BlockNorm, Gate, grouped_gemm_fp8, grouped_wgrad_fp8, quantize_rows, quantize_weights, swiglu_fp8,
               swiglu_fp8_backward)
from .experts import _on


class _NoSecondDerivative(torch.autograd.Function):
    @staticmethod
    def forward(ctx, anchor, what, *grads):
        ctx.what = what
        ctx.set_materialize_grads(False)
        return grads

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.what} has no second derivative")


def _first_order(backward):
    """Marks a backward pass that cannot be differentiated itself.  Under create_graph
    its gradients may be used, but differentiating through them raises, also where the
    incoming gradient is a constant: they depend on the forward pass's inputs."""
    what = backward.__qualname__

    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        out = out if isinstance(out, tuple) else (out,)
        at = [i for i, g in enumerate(out) if g is not None]
        marked = _NoSecondDerivative.apply(torch.empty(0, requires_grad=True), what, *(out[i] for i in at))
        out = list(out)
        for i, g in zip(at, marked):
            out[i] = g
        return tuple(out)

    return run


def _gradient(grad):
    """An incoming gradient as the kernels read it: dense, from a 16-byte boundary (autograd
    hands on views at any offset, a part of a larger tensor's gradient for one)."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


class _Routing:
    """The layout of one dispatch; `handle` is set once dispatch has run."""

    def __init__(self, layout):
        self.layout = layout
        self.handle = None


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, topk_weights, routing, capacity_rows):
        w = topk_weights.detach().contiguous() if topk_weights is not None else None
        recv, _, handle = _dispatch(x.detach().contiguous(), w, routing.layout, False, capacity_rows)
        routing.handle = handle
        ctx.handle = handle
        return recv

    @staticmethod
    @_first_order
    def backward(ctx, grad_recv):
        return _dispatch_backward(_gradient(grad_recv), ctx.handle), None, None, None


def _unmapped_rows_zeroed(y, handle):
    """A gradient buffer shaped like y whose rows that no pair maps to are
    zero (the combine backward writes the others).  In a dense layout whose
    pair count the host has read (handle_recv_counts, which a grouped GEMM
    needs anyway), those rows are exactly [min(N, capacity), rows); otherwise
    every row is zeroed first."""
    c = handle.c
    dense = c.static_cap == 0 and c.expert_alignment <= 1
    if not dense or handle.num_recv is None:
        return torch.zeros_like(y, memory_format=torch.contiguous_format)
    grad_y = torch.empty_like(y, memory_format=torch.contiguous_format)
    grad_y[min(handle.num_recv, c.capacity_rows):].zero_()
    return grad_y


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, topk_weights, handle):
        w = topk_weights.detach().contiguous() if topk_weights is not None else None
        out = _combine(y.detach().contiguous(), handle, w)
        ctx.handle = handle
        ctx.save_for_backward(y, topk_weights)
        return out

    @staticmethod
    @_first_order
    def backward(ctx, grad_out):
        y, w = ctx.saved_tensors
        want_w = w is not None and ctx.needs_input_grad[1]
        grad_y = _unmapped_rows_zeroed(y, ctx.handle)
        gy, gw = _combine_backward(_gradient(grad_out), ctx.handle,
                                   y=y.detach().contiguous() if want_w else None,
                                   topk_weights=w.detach().contiguous() if w is not None else None,
                                   grad_y=grad_y)
        return gy, (gw if want_w else None), None


def dispatch(x, topk_idx, topk_weights, num_experts: int, num_partitions: int,
             capacity_rows=None):
    """BF16 dispatch with a gradient for x.  Returns (recv [capacity, H] bf16,
    handle); ep.handle_recv_counts(handle) gives the per-expert counts."""
    routing = _Routing(_get_dispatch_layout(topk_idx, num_experts, num_partitions))
    recv = _Dispatch.apply(x, topk_weights, routing, capacity_rows)
    return recv, routing.handle


def combine(y, handle, topk_weights=None):
    """Combine with gradients for y and, when it requires grad, topk_weights
    (None: the weights dispatch copied, as constants)."""
    return _Combine.apply(y, topk_weights, handle)


def _eager_only(what):
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{what} cannot be captured into a graph: capture the plain calls instead")


class _Gate(torch.autograd.Function):
    # ctx holds no output but through save_for_backward: a node that holds its own
    # outputs, which hold the node, is never freed
    @staticmethod
    def forward(ctx, logits, num_topk, options, out):
        g = _gate_call(logits.detach(), num_topk, **options)
        out.append(g)
        ctx.save_for_backward(logits, g.topk_idx, g.num_tokens_per_expert, g.num_valid, g.token_mask)
        ctx.options = g.score, g.normalize, g.scale, g.balance_coef
        ctx.mark_non_differentiable(g.topk_idx, g.num_tokens_per_expert)
        ctx.set_materialize_grads(False)
        return g.topk_weights, g.loss, g.topk_idx, g.num_tokens_per_expert

    @staticmethod
    @_first_order
    def backward(ctx, grad_weights, grad_loss, *_):
        _eager_only("the backward pass of gate")
        logits, idx, counts, valid, mask = ctx.saved_tensors
        if grad_weights is not None:
            grad_weights = grad_weights.contiguous()
        if grad_loss is not None:
            grad_loss = grad_loss.contiguous()
        g = Gate(idx, None, counts, valid, None, *ctx.options, mask)
        return _gate_backward(logits.detach(), g, grad_weights, grad_loss), None, None, None


def gate(logits, num_topk: int, **options):
    """The gate (same options) with gradients of its weights and its balance loss
    towards the logits.  Backward reads the logits, ids, counts, num_valid and
    token_mask again: changing one of them in place before is an error."""
    with _on(logits):
        _eager_only("gate")
        kept = []
        w, loss, _, _ = _Gate.apply(logits, num_topk, options, kept)
    return dataclasses.replace(kept[0], topk_weights=w, loss=loss)


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, topk_weights, w1, w2, layout, grad_enabled):
        # inputs that need a gradient count under no_grad too; `inner`: the gradient passes SwiGLU
        want_x, want_w, want_1, want_2 = (grad_enabled and n for n in ctx.needs_input_grad[:4])
        inner = want_x or want_1
        x8, xs, h = _dispatch(x.detach().contiguous(), topk_weights.detach().contiguous(), layout, True)
        q1 = quantize_weights(w1.detach().contiguous(), transposed=want_x)
        q2 = quantize_weights(w2.detach().contiguous(), transposed=inner)
        y1 = grouped_gemm_fp8(x8, xs, q1.codes, q1.scales, h)
        a8, a_s, c8, cs = swiglu_fp8(y1, h, checkpoint=inner)
        y2 = grouped_gemm_fp8(a8, a_s, q2.codes, q2.scales, h)
        ctx.handle = h
        ctx.dtypes = w1.dtype, w2.dtype
        ctx.save_for_backward(*((x8, xs) if want_1 else (None, None)), *((a8, a_s) if want_2 else (None, None)),
                              c8, cs, y2 if want_w else None, q1.codes_t, q1.scales_t, q2.codes_t, q2.scales_t)
        return _combine(y2, h)

    @staticmethod
    @_first_order
    def backward(ctx, grad_out):
        _eager_only("the backward pass of experts")
        x8, xs, a8, a_s, c8, cs, y2, w1t, s1t, w2t, s2t = ctx.saved_tensors
        h = ctx.handle
        want_x, want_w, want_1, want_2 = ctx.needs_input_grad[:4]
        # with dispatch's copy of the weights
        gy, gw = _combine_backward(_gradient(grad_out), h, y=y2 if want_w else None)
        gx = g1 = g2 = None
        if want_2:
            g2 = grouped_wgrad_fp8(gy, a8, a_s, h, out_dtype=ctx.dtypes[1])
        if want_x or want_1:
            g8, gs = quantize_rows(gy, h)
            ga = grouped_gemm_fp8(g8, gs, w2t, s2t, h)
            gh, gh8, ghs = swiglu_fp8_backward(ga, c8, cs, h, quantize=want_x)
            if want_1:
                g1 = grouped_wgrad_fp8(gh, x8, xs, h, out_dtype=ctx.dtypes[0])
            if want_x:
                gx = _dispatch_backward(grouped_gemm_fp8(gh8, ghs, w1t, s1t, h), h)
        return gx, (gw if want_w else None), g1, g2, None, None


def experts(x, topk_idx, topk_weights, w1, w2, num_partitions: int = 1):
    """One expert layer in FP8 with gradients for x, topk_weights, w1 and w2.
    x: bf16 [T, H]; topk_idx, topk_weights: [T, K]; w1: bf16 or fp32 [E, 2 * I, H]
    (gate rows, then up rows), w2: [E, H, I].  Returns bf16 [T, H].  H and I are
    multiples of 128."""
    if not (x.dim() == 2 and topk_idx.dim() == 2 and topk_idx.shape[0] == x.shape[0] and
            topk_weights.shape == topk_idx.shape):
        raise ValueError(f"x [T, H], topk_idx [T, K] and topk_weights [T, K] do not fit: {list(x.shape)}, "
                         f"{list(topk_idx.shape)}, {list(topk_weights.shape)}")
    E, H = w1.shape[0], x.shape[1]
    if not (w1.dim() == 3 and w2.dim() == 3 and w1.shape[1:] == (2 * w2.shape[2], H) and w2.shape[:2] == (E, H)):
        raise ValueError(f"x [T, H], w1 [E, 2 * I, H] and w2 [E, H, I] do not fit: {list(x.shape)}, "
                         f"{list(w1.shape)}, {list(w2.shape)}")
    with _on(x, topk_idx, topk_weights, w1, w2):
        _eager_only("experts")
        layout = _get_dispatch_layout(topk_idx, E, num_partitions)
        # inside forward gradients are always off
        return _Experts.apply(x, topk_weights, w1, w2, layout, torch.is_grad_enabled())


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, weight, y_weight, gate, options):
        # the inputs alone are kept: backward computes both norms' factors again
        inputs = x, y, weight, y_weight, gate
        ctx.save_for_backward(*inputs)
        ctx.options = options
        ctx.set_materialize_grads(False)
        x, y, weight, y_weight, gate = (None if t is None else t.detach() for t in inputs)
        n = _block_norm_call(x, y, weight=weight, y_weight=y_weight, gate=gate, **options)
        return (None if y is None else n.x), n.h

    @staticmethod
    @_first_order
    def backward(ctx, grad_x, grad_h):
        _eager_only("the backward pass of block_norm")
        need = [n for n, wanted in zip(_NORM_INPUTS, ctx.needs_input_grad) if wanted]
        inputs = {n: None if t is None else t.detach() for n, t in zip(_NORM_INPUTS, ctx.saved_tensors)}
        g = _block_norm_backward(grad_x=None if grad_x is None else _gradient(grad_x),
                                 grad_h=None if grad_h is None else _gradient(grad_h),
                                 need=need, **inputs, **ctx.options)
        return (*(getattr(g, n) for n in _NORM_INPUTS), None)


_NORM_INPUTS = ("x", "y", "weight", "y_weight", "gate")


def block_norm(x, y=None, *, norm: bool = True, weight=None, y_norm: bool = False, y_weight=None, gate=None,
               residual_scale: float = 1.0, y_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0):
    """The norms before and after a block (the plain call's arguments, without its 8-bit
    rows: ``experts`` makes its own) with gradients for x, y, weight, y_weight and gate.
    Returns ``BlockNorm``: the new residual stream (x itself without y) and its norm (None
    without norm).  The inputs are kept for backward: changing one of them in place
    before is an error."""
    options = dict(norm=norm, y_norm=y_norm, residual_scale=residual_scale, y_scale=y_scale, eps=eps,
                   weight_offset=weight_offset)
    with _on(x, y, weight, y_weight, gate):
        _eager_only("block_norm")
        x_out, h = _BlockNorm.apply(x, y, weight, y_weight, gate, options)
    return BlockNorm(x if y is None else x_out, h)
