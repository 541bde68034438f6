"""Layers of experts on the library's operators: differentiable wrappers over
the grouped products, the sort of tokens by expert with its way there and back,
and the norm; and the forms for serving in 8 and 4 bits, which have no
gradient.  Rows (tokens, residuals, a token's weights) may have any strides: those
that the library does not take are copied.  A product's weights are not."""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _native as agg

__all__ = ["grouped_linear", "quantize", "quantize_weights", "grouped_linear_fp8",
           "Routing", "sort_by_expert", "dispatch", "combine", "rms_norm", "rms_norm_fp8",
           "quantize_mxfp4", "dequantize_mxfp4", "linear_mxfp4", "grouped_linear_mxfp4"]


def _rows(t):
    """t as the library takes a matrix: unit column stride, rows that do not overlap.
    What is not a matrix stays as it is, for the library's own check."""
    if t is None or t.dim() != 2 or (t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        return t
    return t.contiguous() if t.numel() else t.new_empty(t.shape)     # no values: contiguous as it is


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, trans_w, padded):
        x = _rows(x)
        ctx.save_for_backward(x, w, offsets)
        ctx.trans_w, ctx.padded = trans_w, padded
        make = torch.zeros if padded else torch.empty
        y = make(x.shape[0], w.shape[1 if trans_w else 2], dtype=x.dtype, device=x.device)
        return agg.ag_gemm_grouped(x, w, offsets, y, trans_w)

    @staticmethod
    @once_differentiable     # the gradients' own kernels are not recorded
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = _rows(dy)
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
        raise _no_gradient()


def _no_gradient():
    return RuntimeError("products and quantisers of 8 and 4 bits have no gradient: train with grouped_linear and "
                        "rms_norm, or call them on detached inputs or under no_grad()")


def _wants_gradient(*inputs):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs)


def _serving(call, *inputs):
    if _wants_gradient(*inputs):
        return _Serving.apply(call, *inputs)
    return call(*inputs)


def quantize(x):
    """E4M3 codes of x [M, K] and a fp32 scale for each row and 128 of k (no
    gradient: a backward pass through them is refused)."""
    return _serving(_quantize, x)


def _quantize(x):
    x = _rows(x)
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty(x.shape[0], -(-x.shape[1] // agg.SCALE_BLOCK), dtype=torch.float32, device=x.device)
    return agg.ag_gemm_quant_fp8_block(x, q, scale, 1)


def quantize_weights(w):
    """E4M3 codes of w ([N, K] or [E, N, K]) and a fp32 scale for each 128 x 128
    block (no gradient, as quantize)."""
    return _serving(_quantize_weights, w)


def _quantize_weights(w):
    if w.dim() == 2:
        w = _rows(w)
        q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
        scale = torch.empty(-(-w.shape[0] // agg.SCALE_BLOCK), -(-w.shape[1] // agg.SCALE_BLOCK),
                            dtype=torch.float32, device=w.device)
        return agg.ag_gemm_quant_fp8_block(w, q, scale, agg.SCALE_BLOCK)
    parts = [_quantize_weights(m) for m in w]
    return (torch.stack([q.view(torch.uint8) for q, _ in parts]).view(torch.float8_e4m3fn),
            torch.stack([s for _, s in parts]))


def grouped_linear_fp8(x, wq, w_scale, offsets, out_dtype=None, padded: bool = False):
    """x [T, K] (16-bit, quantised here; or its codes and scales as a pair, with
    the type of the result in ``out_dtype``) times each group's [N, K] E4M3
    weights (no gradient, as quantize).

    The groups cover every row unless ``padded`` is set: rows of no group then
    get zeros."""
    if isinstance(x, (tuple, list)):
        q, scale = x
        return _serving(lambda *operands: _grouped_fp8(*operands, offsets, out_dtype, padded),
                        q, scale, wq, w_scale)

    def call(x, wq, w_scale):
        return _grouped_fp8(*_quantize(x), wq, w_scale, offsets, out_dtype or x.dtype, padded)

    return _serving(call, x, wq, w_scale)


def _grouped_fp8(q, scale, wq, w_scale, offsets, dtype, padded):
    if dtype is None:
        raise ValueError("codes have no type of their own for the result: give out_dtype")
    y = (torch.zeros if padded else torch.empty)(q.shape[0], wq.shape[1], dtype=dtype, device=q.device)
    return agg.ag_gemm_grouped_fp8_block(q, scale, wq, w_scale, offsets, y)


# ---- tokens to their experts and back ---------------------------------------


class Routing(NamedTuple):
    """Where tokens go: row place[t, j] among the rows sorted by expert (-1:
    none), offsets[e] .. offsets[e + 1] the rows of expert e."""

    offsets: torch.Tensor    # int32 [experts + 1]
    place: torch.Tensor      # int32 [T, top]


def sort_by_expert(ids, experts: int) -> Routing:
    """The Routing of ids [T, top] (int32 or int64) by a stable sort; ids outside
    [0, experts) have no place."""
    if ids.dim() != 2:
        raise ValueError("ids must be [T, top]")
    ids = _rows(ids)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device)
    place = torch.empty(ids.shape, dtype=torch.int32, device=ids.device)
    need = agg.expert_sort_workspace_bytes(*ids.shape, experts)
    ws = torch.empty(need, dtype=torch.uint8, device=ids.device) if need else None
    return Routing(*agg.ag_gemm_expert_sort(ids, experts, offsets, place, ws))


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, place, padded):
        ctx.save_for_backward(place)
        xs = (torch.zeros if padded else torch.empty)(place.numel(), x.shape[1], dtype=x.dtype, device=x.device)
        return agg.ag_gemm_expert_dispatch(_rows(x), place, xs)

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        place, = ctx.saved_tensors
        dxs = _rows(dxs)
        dx = torch.empty(place.shape[0], dxs.shape[1], dtype=dxs.dtype, device=dxs.device)
        return agg.ag_gemm_expert_combine(dxs, place, None, dx), None, None


def dispatch(x, routing: Routing, padded: bool = False):
    """Rows of x [T, K] (or codes and their scales, each on its own) in the order
    of the experts, [T * top, K]; differentiable.

    Every assignment has a place unless ``padded`` is set: the rows behind the
    last place are then zeros."""
    return _Dispatch.apply(x, routing.place, padded)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, weights, place, padded):
        h, weights = _rows(h), _rows(weights)
        ctx.save_for_backward(h, weights, place)
        ctx.padded = padded
        y = torch.empty(place.shape[0], h.shape[1], dtype=h.dtype, device=h.device)
        return agg.ag_gemm_expert_combine(h, place, weights, y)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        h, weights, place = ctx.saved_tensors
        dy = _rows(dy)
        dh = dw = None
        if ctx.needs_input_grad[0]:
            dh = (torch.zeros if ctx.padded else torch.empty)(h.shape, dtype=h.dtype, device=h.device)
        if ctx.needs_input_grad[1]:
            dw = torch.empty(weights.shape, dtype=weights.dtype, device=weights.device)
        if dh is not None or dw is not None:
            agg.ag_gemm_expert_combine_grad(dy, h, place, weights, dh, dw)
        return dh, dw, None, None


def combine(h, weights, routing: Routing, padded: bool = False):
    """y[t] = sum over j of weights[t, j] * h[place[t, j]], differentiable in h
    [T * top, K] and weights [T, top] (summed in fp32, whatever their type).

    Every assignment has a place unless ``padded`` is set: rows of h without one
    then get zeros as their gradient."""
    return _Combine.apply(h, weights.float(), routing.place, padded)


# ---- norm ---------------------------------------------------------------------


def _flat(t, k):
    """t [..., k] as a matrix."""
    return _rows(t.reshape(t.shape[:-1].numel(), k))


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        k = x.shape[-1]
        flat, res = _flat(x, k), None if residual is None else _flat(residual, k)
        weight = None if weight is None else weight.contiguous()
        y = torch.empty(flat.shape, dtype=x.dtype, device=x.device)
        h = None if residual is None else torch.empty_like(y)
        rstd = torch.empty(flat.shape[0], dtype=torch.float32, device=x.device)
        agg.ag_gemm_rmsnorm(flat, weight, y=y, residual=res, h=h, rstd=rstd, eps=eps)
        y, h = y.view(x.shape), None if h is None else h.view(x.shape)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        return y if h is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        wants = ctx.needs_input_grad
        wants_w = weight is not None and wants[1]
        dx, dw, ws = dh, None, None
        if dy is not None:       # else only h was used
            dy, flat = _flat(dy, h.shape[-1]), _flat(h, h.shape[-1])
            dx = torch.empty(flat.shape, dtype=h.dtype, device=h.device)
            if wants_w:
                dw = torch.empty_like(weight)
                ws = torch.empty(agg.rmsnorm_grad_workspace_bytes(*flat.shape), dtype=torch.uint8, device=h.device)
            agg.ag_gemm_rmsnorm_grad(dy, flat, weight, rstd, dx, dw, ws,
                                     None if dh is None else _flat(dh, h.shape[-1]))
            dx = dx.view(h.shape)
        elif wants_w:
            dw = torch.zeros_like(weight)
        # one tensor for both: autograd copies what two leaves would share
        return dx if wants[0] else None, dw, dx if wants[2] else None, None


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6):
    """h / sqrt(mean(h^2) + eps) * weight of the rows of h = x + residual (h = x
    without one), x and residual [..., K] and weight [K] of one type;
    differentiable.  With a residual the result is (y, h): h, rounded to its type,
    is the next residual."""
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual must have x's shape {tuple(x.shape)}")
    return _RmsNorm.apply(x, weight, residual, eps)


def rms_norm_fp8(x, weight=None, residual=None, eps: float = 1e-6, with_y: bool = False):
    """rms_norm's result as E4M3 codes and a fp32 scale for each row and 128
    columns (no gradient, as quantize): x [T, K].  The result is codes, scales, with
    ``with_y`` the values in x's type too (for a router), and with a residual h."""
    def call(x, weight, residual):
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty(x.shape[0], -(-x.shape[1] // agg.SCALE_BLOCK), dtype=torch.float32, device=x.device)
        y, h = (torch.empty(x.shape, dtype=x.dtype, device=x.device) if wanted else None
                for wanted in (with_y, residual is not None))
        agg.ag_gemm_rmsnorm(_rows(x), None if weight is None else weight.contiguous(), y=y, q=q, scale=scale,
                            residual=_rows(residual), h=h, eps=eps)
        return (q, scale, *(t for t in (y, h) if t is not None))

    return _serving(call, x, weight, residual)


# ---- microscaled 4-bit values -------------------------------------------------


def quantize_mxfp4(x):
    """E2M1 codes (two a byte) and E8M0 scales (one for each 32 columns) of x [...,
    K], K even: activations [M, K] or weights [N, K] or [E, N, K].  Both are
    integers, which autograd does not follow: an x that needs a gradient is
    refused (parameters are quantised detached or under no_grad())."""
    if _wants_gradient(x):
        raise _no_gradient()
    k = x.shape[-1]
    flat = _flat(x, k)
    q = torch.empty(flat.shape[0], k // 2, dtype=torch.uint8, device=x.device)
    # rows of scales on 4-byte boundaries, as the faster products take them
    kb = -(-k // agg.MX_BLOCK)
    pitch = -(-kb // 4) * 4
    scale = torch.empty(flat.shape[0], pitch, dtype=torch.uint8, device=x.device)
    agg.ag_gemm_quant_mxfp4(flat, q, scale[:, :kb])
    return q.view(*x.shape[:-1], k // 2), scale.view(*x.shape[:-1], pitch)[..., :kb]


def dequantize_mxfp4(q, scale, dtype=torch.bfloat16):
    """The values of quantize_mxfp4's codes and scales."""
    k, kb = 2 * q.shape[-1], scale.shape[-1]
    y = torch.empty(*q.shape[:-1], k, dtype=dtype, device=q.device)
    agg.ag_gemm_dequant_mxfp4(_flat(q, k // 2), _flat(scale, kb), _flat(y, k))
    return y


def linear_mxfp4(x, wq, w_scale, out_dtype=None):
    """x [M, K] (quantised here) times [N, K] weights of 4 bits, transposed (no
    gradient, as quantize)."""
    def call(x):
        y = torch.empty(x.shape[0], wq.shape[0], dtype=out_dtype or x.dtype, device=x.device)
        return agg.ag_gemm_mxfp4(*quantize_mxfp4(x), wq, w_scale, y)

    return _serving(call, x)


def grouped_linear_mxfp4(x, wq, w_scale, offsets, out_dtype=None, padded: bool = False):
    """x [T, K] (quantised here) times each group's [N, K] weights of 4 bits (no
    gradient, as quantize).

    The groups cover every row unless ``padded`` is set: rows of no group then
    get zeros."""
    def call(x):
        make = torch.zeros if padded else torch.empty
        y = make(x.shape[0], wq.shape[1], dtype=out_dtype or x.dtype, device=x.device)
        return agg.ag_gemm_grouped_mxfp4(*quantize_mxfp4(x), wq, w_scale, offsets, y)

    return _serving(call, x)
