"""A gated feed-forward block of E experts, put together from the package's
operators: router logits [T, E] send each of T tokens to k experts, expert e
maps a row x to W2_e (silu(g) * u) with (g, u) the halves of W1_e x, and the k
results are added with the router's weights.

    ffn_int8   serving: the two products in 8-bit integers
    ffn_mxfp4  serving: the two products in microscaled 4-bit floating point
    ffn        training: BF16 products, differentiable in the rows, the logits
               and both weights; with kept="int8" its backward pass computes
               from 8-bit gate and up rows and keeps no other rows of the experts

Weights are stacked per expert, W1 [E, 2I, H] (gate rows, then up rows) and
W2 [E, H, I].  Derivatives are of first order: a second one through these
operators raises.
"""
import torch

from . import (Routing, Scoring, grouped_gemm_dgrad, grouped_gemm_fwd, grouped_gemm_int8, grouped_gemm_wgrad, moe_combine, moe_combine_grad,
               moe_dispatch, moe_ffn_int8, moe_ffn_mxfp4, moe_gate_int8, moe_gate_int8_grad, moe_route, moe_route_grad,
               moe_route_scores, moe_route_scores_grad, quantize_int8, quantize_mxfp4)
from .autograd import gradient, grouped_linear


def quantize_weights(W):
    """Codes and scales of stacked weights [E, N, K] (BF16 or FP32), one scale
    per expert and output channel: (int8 [E, N, K], FP32 [E, N])."""
    E, N, K = W.shape
    q, scale = quantize_int8(W.reshape(E * N, K))
    return q.view(E, N, K), scale.view(E, N)


def ffn_int8(X, logits, W1q, w1_scale, W2q, w2_scale, k, renormalize=True, scoring=None):
    """The block on 8-bit weights (codes and scales as quantize_weights gives
    them): X [T, H] BF16 to [T, H] BF16.  Rows are quantised per token before
    each product; the activation between the products stays in FP32 until
    then (rounded to BF16 first, values near the border of two codes would
    take the other one, which moves the result by 0.75 % of its norm).  The
    experts' outputs are rounded to BF16 before they are added in FP32.
    scoring: a Scoring to select by scores (renormalize is then the Scoring's),
    by the block's single calls instead of the one."""
    if scoring is None:
        return moe_ffn_int8(X, logits, W1q, w1_scale, W2q, w2_scale, k, renormalize=renormalize)
    r = moe_route_scores(logits, k, scoring)
    gather = X.numel() < 2 ** 31 - 4096
    q, scale = quantize_int8(X) if gather else quantize_int8(X, r.positions)
    h = grouped_gemm_int8(q, scale, W1q, w1_scale, r.group_offsets, gated=True, rows=r.tokens if gather else None,
                          out_dtype=torch.float32)
    y = grouped_gemm_int8(*quantize_int8(h), W2q, w2_scale, r.group_offsets)
    return moe_combine(y, r.positions, r.weights)


def quantize_weights_mxfp4(W):
    """4-bit codes and scales of stacked weights [E, N, K] (BF16 or FP32), a
    scale for each 32 values of a row: (uint8 [E, N, K/2], uint8
    [ceil(K/256), E, N, 8])."""
    E, N, K = W.shape
    codes, scales = quantize_mxfp4(W.reshape(E * N, K))
    return codes.view(E, N, K // 2), scales.view(-1, E, N, 8)


def ffn_mxfp4(X, logits, W1q, w1_scale, W2q, w2_scale, k, scoring=None):
    """The block on 4-bit weights (codes and scales as quantize_weights_mxfp4
    gives them): X [T, H] BF16 to [T, H] BF16.  Rows are quantised to 4 bits
    before each product, the activation from FP32; the experts' outputs are
    rounded to BF16 before they are added in FP32.  scoring: a Scoring, or None
    for the softmax over the k largest logits."""
    return moe_ffn_mxfp4(X, logits, W1q, w1_scale, W2q, w2_scale, k, scoring=scoring)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, renormalize):
        r = moe_route(logits, k, renormalize=renormalize)
        ctx.save_for_backward(logits, r.experts, r.weights)
        ctx.renormalize = renormalize
        ctx.mark_non_differentiable(r.experts, r.group_offsets, r.positions, r.tokens)
        return tuple(r)

    @staticmethod
    def backward(ctx, _experts, dweights, _offsets, _positions, _tokens):
        logits, experts, weights = ctx.saved_tensors
        return gradient(lambda *a: moe_route_grad(*a, renormalize=ctx.renormalize), dweights.contiguous(), logits, experts,
                        weights), None, None


class _RouteScores(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, scoring):
        r = moe_route_scores(logits, k, scoring)
        ctx.save_for_backward(logits, r.experts, r.weights)
        ctx.scoring = scoring._replace(bias=None)   # takes no part in the gradient
        ctx.mark_non_differentiable(r.experts, r.group_offsets, r.positions, r.tokens)
        return tuple(r)

    @staticmethod
    def backward(ctx, _experts, dweights, _offsets, _positions, _tokens):
        logits, experts, weights = ctx.saved_tensors
        return gradient(lambda *a: moe_route_scores_grad(*a, scoring=ctx.scoring), dweights.contiguous(), logits, experts,
                        weights), None, None


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, positions):
        ctx.save_for_backward(positions)
        return moe_dispatch(X, positions)

    @staticmethod
    def backward(ctx, dout):
        return gradient(moe_combine, dout.contiguous(), *ctx.saved_tensors), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, positions, weights):
        ctx.save_for_backward(rows, positions, weights)
        return moe_combine(rows, positions, weights)

    @staticmethod
    def backward(ctx, dout):
        drows, dweights = gradient(moe_combine_grad, dout.contiguous(), *ctx.saved_tensors)
        return drows, None, dweights


class _Experts8(torch.autograd.Function):
    """The experts' part of the block, from token rows to token rows, with the
    pairs' weights applied in the activation: out = combine(h W2^T), h = weight *
    silu(g) * u, (g, u) = dispatch(X) W1^T.  Kept for the backward pass: the
    inputs, and g and u in 8 bits; the dispatched rows, the activation and the
    rows' gradients are made again where they are needed."""

    @staticmethod
    def forward(ctx, X, weights, W1, W2, group_offsets, positions, deterministic):
        GU = grouped_gemm_fwd(moe_dispatch(X, positions), W1, group_offsets)
        h, codes, scale = moe_gate_int8(GU, positions, weights)
        del GU
        ctx.save_for_backward(X, weights, W1, W2, group_offsets, positions, codes, scale)
        ctx.deterministic = bool(deterministic)
        return moe_combine(grouped_gemm_fwd(h, W2, group_offsets), positions)

    @staticmethod
    def backward(ctx, dout):
        need = ctx.needs_input_grad[:4]
        det = ctx.deterministic

        def grads(dout, X, weights, W1, W2, offsets, positions, codes, scale):
            drows = moe_dispatch(dout, positions)
            dh = grouped_gemm_dgrad(drows, W2, offsets)
            dGU, h, dweights = moe_gate_int8_grad(dh, codes, scale, positions, weights)
            del dh
            dW2 = grouped_gemm_wgrad(h, drows, offsets, deterministic=det) if need[3] else None
            del drows, h
            dW1 = grouped_gemm_wgrad(moe_dispatch(X, positions), dGU, offsets, deterministic=det) if need[2] else None
            dX = moe_combine(grouped_gemm_dgrad(dGU, W1, offsets), positions) if need[0] else None
            return dX, dweights if need[1] else None, dW1, dW2
        return (*gradient(grads, dout.contiguous(), *ctx.saved_tensors), None, None, None)


def route(logits, k, renormalize=True):
    """moe_route, differentiable: a Routing whose weights are differentiable in
    the logits."""
    return Routing(*_Route.apply(logits, k, renormalize))


def route_scores(logits, k, scoring=Scoring()):
    """moe_route_scores, differentiable in the logits as route is."""
    return Routing(*_RouteScores.apply(logits, k, scoring))


def dispatch(X, positions):
    """moe_dispatch, differentiable in X."""
    return _Dispatch.apply(X, positions)


def combine(rows, positions, weights):
    """The weighted moe_combine, differentiable in rows and weights."""
    return _Combine.apply(rows, positions, weights)


def ffn(X, logits, W1, W2, k, renormalize=True, deterministic=True, scoring=None, kept=None):
    """The block in BF16, differentiable in X [T, H], logits [T, E] (FP32), W1
    and W2; the weight gradients as autograd.grouped_linear computes them.  What
    passes from one operator to the next is BF16: gate and up, silu(gate), its
    product with up, and the experts' outputs are rounded once each.

    scoring: a Scoring to select by scores; renormalize is then the Scoring's.
    kept="int8": gate and up are kept in 8 bits (a scale for each 128 columns)
    and the backward pass computes from them; of the experts' T*k rows nothing
    else is kept (without it: the dispatched rows, gate and up, silu(gate), the
    activation and the experts' outputs).  The pairs' weights are applied to the
    activation, in FP32 before its one rounding."""
    r = route(logits, k, renormalize) if scoring is None else route_scores(logits, k, scoring)
    if kept == "int8":
        return _Experts8.apply(X, r.weights, W1, W2, r.group_offsets, r.positions, deterministic)
    if kept is not None:
        raise ValueError(f"kept={kept!r}: int8 or None")
    gate, up = grouped_linear(dispatch(X, r.positions), W1, r.group_offsets, deterministic).chunk(2, dim=1)
    h = torch.nn.functional.silu(gate) * up
    return combine(grouped_linear(h, W2, r.group_offsets, deterministic), r.positions, r.weights)
