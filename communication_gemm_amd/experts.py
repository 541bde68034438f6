"""Layers of experts on the grouped products: differentiable wrappers over
ag_gemm_grouped and ag_gemm_grouped_wgrad, and the fp8 form for serving."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _native as agg

__all__ = ["grouped_linear", "quantize", "quantize_weights", "grouped_linear_fp8"]


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, trans_w, padded):
        ctx.save_for_backward(x, w, offsets)
        ctx.trans_w, ctx.padded = trans_w, padded
        make = torch.zeros if padded else torch.empty
        y = make(x.shape[0], w.shape[1 if trans_w else 2], dtype=x.dtype, device=x.device)
        return agg.ag_gemm_grouped(x, w, offsets, y, trans_w)

    @staticmethod
    @once_differentiable     # the gradients' own kernels are not recorded
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        if dy.stride(-1) != 1 or dy.stride(0) < dy.shape[1]:
            dy = dy.contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = (torch.zeros if ctx.padded else torch.empty)(x.shape, dtype=x.dtype, device=x.device)
            agg.ag_gemm_grouped(dy, w, offsets, dx, not ctx.trans_w)
        if ctx.needs_input_grad[1]:
            dw = torch.empty(w.shape, dtype=w.dtype, device=w.device)
            a, b = (dy, x) if ctx.trans_w else (x, dy)
            agg.ag_gemm_grouped_wgrad(a, b, offsets, dw)
        return dx, dw, None, None, None


def grouped_linear(x, w, offsets, trans_w: bool = False, padded: bool = False):
    """y[r] = x[r] @ w[e(r)], differentiable in x [T, K] and w [E, K, N] (with
    trans_w [E, N, K]); offsets int32 [E + 1].

    The groups cover every row unless ``padded`` is set: rows of no group then
    get zeros in y and in x's gradient."""
    return _GroupedLinear.apply(x, w, offsets, trans_w, padded)


class _Serving(torch.autograd.Function):
    """A call that no gradient passes through: asking for one is an error,
    where leaving it out would train on without it."""

    @staticmethod
    def forward(ctx, call, *inputs):
        ctx.set_materialize_grads(False)
        return call(*inputs)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the fp8 product and its quantiser have no gradient: train with "
                           "grouped_linear, or call them on detached inputs or under no_grad()")


def _serving(call, *inputs):
    if torch.is_grad_enabled() and any(t.requires_grad for t in inputs):
        return _Serving.apply(call, *inputs)
    return call(*inputs)


def quantize(x):
    """E4M3 codes of x [M, K] and a fp32 scale for each row and 128 of k (no
    gradient: a backward pass through them is refused)."""
    return _serving(_quantize, x)


def _quantize(x):
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty(x.shape[0], -(-x.shape[1] // agg.SCALE_BLOCK), device=x.device)
    return agg.ag_gemm_quant_fp8_block(x, q, scale, 1)


def quantize_weights(w):
    """E4M3 codes of w ([N, K] or [E, N, K]) and a fp32 scale for each 128 x 128
    block (no gradient, as quantize)."""
    return _serving(_quantize_weights, w)


def _quantize_weights(w):
    if w.dim() == 2:
        q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
        scale = torch.empty(-(-w.shape[0] // agg.SCALE_BLOCK), -(-w.shape[1] // agg.SCALE_BLOCK),
                            device=w.device)
        return agg.ag_gemm_quant_fp8_block(w, q, scale, agg.SCALE_BLOCK)
    parts = [_quantize_weights(m) for m in w]
    return (torch.stack([q.view(torch.uint8) for q, _ in parts]).view(torch.float8_e4m3fn),
            torch.stack([s for _, s in parts]))


def grouped_linear_fp8(x, wq, w_scale, offsets, out_dtype=None, padded: bool = False):
    """x [T, K] (16-bit, quantised here) times each group's [N, K] E4M3 weights
    (no gradient, as quantize).

    The groups cover every row unless ``padded`` is set: rows of no group then
    get zeros."""
    def call(x, wq, w_scale):
        make = torch.zeros if padded else torch.empty
        y = make(x.shape[0], wq.shape[1], dtype=out_dtype or x.dtype, device=x.device)
        q, scale = _quantize(x)
        return agg.ag_gemm_grouped_fp8_block(q, scale, wq, w_scale, offsets, y)

    return _serving(call, x, wq, w_scale)
